"""The oracle of the operators beside the layer forward: packing against the codecs, the
gradients against central differences, and degenerate rows."""
import numpy as np
import pytest

from oracle import codecs as OC
from oracle import ops as OP


@pytest.mark.parametrize("K", [32, 96, 256])
def test_int4_unpack_inverts_pack(K):
    q = np.random.default_rng(K).integers(-7, 8, (2, 5, K)).astype(np.int8)
    np.testing.assert_array_equal(OP.int4_unpack(OC.int4_pack(q)), q)
    assert OP.int4_unpack(np.full((1, 4), 0x88, np.uint8)).max() == 0


def test_int4_quant_group_of_128_is_the_codecs():
    w = np.random.default_rng(1).standard_normal((2, 3, 256)).astype(np.float32)
    for a, b in zip(OP.int4_quant_group(w, 128), OC.int4_quant_rows(w)):
        np.testing.assert_array_equal(a, b)


def _router(T, E, k, seed):
    r = np.random.default_rng(seed)
    z = r.standard_normal((T, E)).astype(np.float32)
    idx = np.argsort(-z, axis=1)[:, :k].astype(np.int32)
    return r, z, idx


@pytest.mark.parametrize("kind", ["switch", "square"])
@pytest.mark.parametrize("offsets", [None, [0, 5, 5, 12]])
def test_balance_gradient_against_differences(kind, offsets):
    """L is smooth in the logits with the counts held, so central differences of step h
    (a power of two, exact in fp32 here) are off by O(h^2): at most h^2 sum|terms| ~ 1e-4 of
    the largest gradient."""
    T, E, k, h = 14, 6, 2, 2.0 ** -7
    r, z, idx = _router(T, E, k, 3)
    z = (np.round(z * 64) / 64).astype(np.float32)
    mask = (r.random(T) < 0.8).astype(np.uint8)
    _, _, _, g = OP.balance_loss(z, idx, mask=mask, offsets=offsets, coef=1.0, kind=kind)
    dz, _ = OP.route_bwd(z, idx, mask=mask, offsets=offsets, balance_grad=g, dloss=1.0)
    got = np.zeros_like(dz)
    for t in range(T):
        for e in range(E):
            up, down = z.copy(), z.copy()
            up[t, e] += h
            down[t, e] -= h
            a, b = (OP.balance_loss(v, idx, mask=mask, offsets=offsets, coef=1.0, kind=kind)[0]
                    for v in (up, down))
            got[t, e] = (a - b) / (2 * h)
    assert np.max(np.abs(got - dz)) <= 4 * h * h * np.max(np.abs(dz))


@pytest.mark.parametrize("renorm", [False, True])
def test_gate_gradient_against_differences(renorm):
    T, E, k, h = 9, 7, 3, 2.0 ** -7
    r, z, idx = _router(T, E, k, 4)
    z = (np.round(z * 64) / 64).astype(np.float32)
    idx[2, 1] = idx[2, 0]                    # the same expert twice
    idx[3, 2] = -1                           # a dropped slot
    idx[4] = -1                              # a token without experts
    dw = r.standard_normal((T, k))
    dz, mag = OP.route_bwd(z, idx, dtopk_w=dw, renorm=renorm)
    assert np.all(dz[4] == 0)
    ok = idx >= 0
    got = np.zeros_like(dz)
    for t in range(T):
        for e in range(E):
            f = []
            for s in (h, -h):
                v = z.copy()
                v[t, e] += s
                f.append(np.sum(np.where(ok, OP.gate_weights(v, idx, None, renorm)[0] * dw, 0)))
            got[t, e] = (f[0] - f[1]) / (2 * h)
    assert np.max(np.abs(got - dz)) <= 4 * h * h * np.max(mag)


def test_rows_without_experts_or_tokens():
    z = np.full((4, 3), -np.inf, np.float32)
    idx = np.zeros((4, 1), np.int32)
    loss, counts, probs, grad = OP.balance_loss(z, idx)
    assert np.all(probs == 0) and loss == 0 and counts[0].tolist() == [4, 0, 0]
    dz, _ = OP.route_bwd(z, idx, dtopk_w=np.ones((4, 1)))
    assert np.all(dz == 0)
    loss, counts, probs, grad = OP.balance_loss(z, idx, mask=np.zeros(4, np.uint8))
    assert loss == 0 and counts.sum() == 0 and np.all(grad == 0)
