"""GPU parity of the operators of include/moe_ops.h against the fp64 oracle.

Tolerances are counted from the arithmetic: u = 2^-24 is half a step of fp32 relative to the
value, an addition that truncates is off by 2 u, and an output type adds half its own step.
"""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_amd as M
from oracle import codecs as OC
from oracle import ops as OP
from gpu_util import dev, note, to_np

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}   # rounding, relative to the value


def gen(seed):
    return np.random.default_rng(seed)


def t_(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(dev())


def weights(r, G, rows, K, group):
    q = r.integers(-7, 8, (G, rows, K)).astype(np.int8)
    s = ((0.5 + r.random((G, rows, K // group))) / (4.5 * K ** 0.5)).astype(np.float32)
    return OC.int4_pack(q), s


def rows(r, n, K, dtype):
    x = t_(r.standard_normal((n, K)).astype(np.float32), dtype)
    return x, to_np(x).astype(np.float64)


def sum_error(absum, K, group):
    """Bound of the fp32 sums: any order inside a group, then any order over the groups (and
    over at most 16 partial sums), one rounding of the scale's product each, 2 u a step."""
    return 2 * U * (group + K // group + 17) * absum


def swiglu(v, err):
    """silu(gate) * up of [S, 2N] and its error from those of the products; exp, divide and
    the two multiplications are off by at most 8 u together, and 2 u |z| from exp's
    argument."""
    N = v.shape[1] // 2
    g, u, dg, du = v[:, :N], v[:, N:], err[:, :N], err[:, N:]
    sig = 0.5 * (1 + np.tanh(0.5 * g))
    s, ds = g * sig, np.abs(sig * (1 + g * (1 - sig)))
    h = s * u
    # the slope of silu changes by at most 1/2 per unit of its argument
    dh = (ds + 0.5 * dg) * dg * (np.abs(u) + du) + np.abs(s) * du
    return h, dh + (8 + 2 * np.abs(g)) * U * np.abs(h)


def check(y, ref, err):
    y64 = to_np(y).astype(np.float64)
    tol = err + HALF[y.dtype] * (np.abs(ref) + err)
    bad = ~(np.abs(y64 - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float(np.max(np.abs(y64 - ref) - tol)))


# ------------------------------------------------------------------ quantiser

@pytest.mark.parametrize("shape, group", [((1, 1, 32), 32), ((2, 5, 96), 32), ((3, 7, 192), 64),
                                          ((2, 33, 384), 128)])
def test_quant_group_bitexact(shape, group):
    note(f"quant group {shape} {group}")
    w = (gen(1).standard_normal(shape) * 0.02).astype(np.float32)
    w[0, 0, :group] = 0
    q, s = M.moe_quant_weight_int4_group(t_(w), group)
    qo, so = OP.int4_quant_group(w, group)
    np.testing.assert_array_equal(to_np(q), OC.int4_pack(qo))
    np.testing.assert_array_equal(to_np(s), so)


def test_quant_group_of_128_is_the_128_quantiser():
    note("quant group 128")
    w = t_((gen(2).standard_normal((2, 40, 512)) * 0.02).astype(np.float32))
    for a, b in zip(M.moe_quant_weight_int4_group(w, 128), M.moe_quant_weight_int4(w)):
        assert torch.equal(a, b)


# --------------------------------------------------------------------- matvec

SIZES = [  # S, N, K, group
    (1, 1, 32, 32), (1, 16, 128, 128), (1, 17, 64, 64), (2, 15, 96, 32), (3, 33, 160, 32),
    (1, 100, 2048, 128), (5, 1003, 4128, 32), (16, 48, 192, 64), (17, 31, 256, 128),
    (40, 20, 320, 64), (4, 7, 16384, 128), (1, 515, 7168, 128), (16, 40, 7168, 64),
]


@pytest.mark.parametrize("S, N, K, group", SIZES)
@pytest.mark.parametrize("x_dt", ["bf16", "f32"])
@pytest.mark.parametrize("epi", ["plain", "swiglu"])
def test_matvec_dense(S, N, K, group, x_dt, epi):
    note(f"matvec dense S={S} N={N} K={K} group={group} {x_dt} {epi}")
    r = gen(S * 1000 + N)
    nb = 2 * N if epi == "swiglu" else N
    q, s = weights(r, 1, nb, K, group)
    x, x64 = rows(r, S, K, DT[x_dt])
    v, absum = OP.matvec_int4(x64, OP.int4_weight(q, s), None, 1)
    err = sum_error(absum, K, group)
    if epi == "swiglu":
        v, err = swiglu(v, err)
    for out in (torch.float32, torch.bfloat16):
        y = M.moe_matvec_int4(x, t_(q), t_(s), swiglu=epi == "swiglu", out_dtype=out)
        assert y.dtype == out and tuple(y.shape) == (S, N)
        check(y, v, err)


@pytest.mark.parametrize("T, k, G, N, K, group", [
    (1, 2, 4, 24, 256, 128), (3, 2, 2, 40, 128, 64), (7, 3, 300, 17, 96, 32),
    (40, 4, 5, 33, 192, 64), (128, 8, 16, 8, 128, 128), (1, 8, 8, 16, 2080, 32),
])
@pytest.mark.parametrize("x_dt", ["bf16", "f32"])
@pytest.mark.parametrize("epi", ["plain", "swiglu"])
def test_matvec_routed(T, k, G, N, K, group, x_dt, epi):
    """Slots in any order, several per expert, the same expert twice in a token, and experts
    outside [0, G)."""
    note(f"matvec routed T={T} k={k} G={G} N={N} K={K} group={group} {x_dt} {epi}")
    r = gen(T * 100 + G)
    nb = 2 * N if epi == "swiglu" else N
    q, s = weights(r, G, nb, K, group)
    idx = r.integers(0, G, T * k).astype(np.int32)
    idx[::5] = [-1, G, 2 ** 31 - 1, -2 ** 31][T % 4]
    x, x64 = rows(r, T, K, DT[x_dt])
    v, absum = OP.matvec_int4(x64, OP.int4_weight(q, s), idx, k)
    err = sum_error(absum, K, group)
    if epi == "swiglu":
        v, err = swiglu(v, err)
    y = M.moe_matvec_int4(x, t_(q), t_(s), t_(idx), x_div=k, swiglu=epi == "swiglu",
                          out_dtype=torch.float32)
    check(y, v, err)
    out = (idx < 0) | (idx >= G)
    assert np.all(to_np(y)[out] == 0)


@pytest.mark.parametrize("T, k, G, N, K, group", [
    # passes of 48 rows: all of a matrix, and experts with uneven numbers of slots
    (200, 0, 1, 2001, 160, 32), (64, 0, 1, 8200, 192, 64), (130, 0, 1, 2600, 1152, 128),
    (64, 4, 2, 2500, 96, 32), (170, 6, 5, 1300, 320, 64), (49, 1, 1, 10300, 128, 128),
])
@pytest.mark.parametrize("x_dt", ["bf16", "f32"])
@pytest.mark.parametrize("epi", ["plain", "swiglu"])
def test_matvec_many_slots_an_expert(T, k, G, N, K, group, x_dt, epi):
    note(f"matvec many T={T} k={k} G={G} N={N} K={K} group={group} {x_dt} {epi}")
    r = gen(T + N)
    nb = 2 * N if epi == "swiglu" else N
    q, s = weights(r, G, nb, K, group)
    x, x64 = rows(r, T, K, DT[x_dt])
    idx = None
    if k:
        # the first expert gets most slots; some get none
        idx = np.minimum(r.integers(-1, 2 * G, T * k), G - 1).astype(np.int32)
    v, absum = OP.matvec_int4(x64, OP.int4_weight(q, s), idx, max(k, 1))
    err = sum_error(absum, K, group)
    if epi == "swiglu":
        v, err = swiglu(v, err)
    y = M.moe_matvec_int4(x, t_(q), t_(s), None if idx is None else t_(idx), x_div=max(k, 1),
                          swiglu=epi == "swiglu", out_dtype=torch.float32)
    check(y, v, err)


def test_matvec_1024_slots_of_one_expert():
    note("matvec 1024 slots")
    r = gen(9)
    S, N, K = 1024, 20, 64
    q, s = weights(r, 3, N, K, 32)
    x, x64 = rows(r, S, K, torch.bfloat16)
    idx = np.full(S, 2, np.int32)
    v, absum = OP.matvec_int4(x64, OP.int4_weight(q, s), idx, 1)
    check(M.moe_matvec_int4(x, t_(q), t_(s), t_(idx)), v, sum_error(absum, K, 32))


def test_matvec_keeps_what_it_must_not_touch():
    """Values of rows that no slot uses, NaN and infinities of other slots' rows and experts,
    and the bytes around the output do not reach it."""
    note("matvec isolation")
    r = gen(10)
    G, N, K = 4, 19, 160
    q, s = weights(r, G, N, K, 32)
    s[3] = np.nan                                   # expert 3 is never chosen
    x, _ = rows(r, 6, K, torch.float32)
    x[1] = float("nan")
    x[2, 5] = float("inf")
    idx = np.array([0, -1, 1, 2, 0, 1], np.int32)
    y = M.moe_matvec_int4(x, t_(q), t_(s), t_(idx))
    alone = torch.cat([M.moe_matvec_int4(x[i:i + 1].clone(), t_(q), t_(s), t_(idx[i:i + 1]))
                       for i in range(6)])
    assert torch.equal(y[[0, 3, 4, 5]], alone[[0, 3, 4, 5]])
    assert torch.isfinite(y[[0, 3, 4, 5]]).all() and torch.all(y[1] == 0)
    assert not torch.isfinite(y[2]).any()
    room = torch.full((8, N), 7.0, device=dev())
    lib_out = room[1:7]
    from fp8_grouped_gemm_amd import _lib
    import ctypes as C
    p = lambda t: C.c_void_p(t.data_ptr())  # noqa: E731
    tq, ts, ti = t_(q), t_(s), t_(idx)
    _lib.check(_lib.load().moe_matvec_int4(p(x), _lib.MOE_F32, 1, p(tq), p(ts), 32, p(ti), 6, G, N,
                                           K, 0, p(lib_out), _lib.MOE_F32,
                                           C.c_void_p(torch.cuda.current_stream().cuda_stream)),
               "moe_matvec_int4")
    torch.cuda.synchronize()
    assert torch.all(room[0] == 7) and torch.all(room[7] == 7)
    assert torch.equal(room[1], y[0])


def test_matvec_f32_rows_of_any_magnitude():
    """fp32 rows whose values need all 24 bits and span many powers of two."""
    note("matvec f32 magnitudes")
    r = gen(12)
    K, N = 256, 50
    q, s = weights(r, 1, N, K, 64)
    x = (r.standard_normal((3, K)) * np.exp2(r.integers(-40, 40, (3, K)))).astype(np.float32)
    x[2] = (r.standard_normal(K) * 3e36).astype(np.float32)
    s[0] *= np.float32(1e-3)
    v, absum = OP.matvec_int4(x, OP.int4_weight(q, s), None, 1)
    check(M.moe_matvec_int4(t_(x), t_(q), t_(s)), v, sum_error(absum, K, 64))


# ------------------------------------------------------------------------ FFN

def ffn_oracle(x64, w13, w2, idx, gw, K, I, group):
    T, k = idx.shape
    E = w13.shape[0]
    flat = idx.ravel()
    v, a = OP.matvec_int4(x64, w13, flat, k)
    h, dh = swiglu(v, sum_error(a, K, group))
    o, oa = OP.matvec_int4(h, w2, flat, 1)
    _, more = OP.matvec_int4(dh + U * np.abs(h), w2, flat, 1)
    do = more + sum_error(oa + more, I, group)
    ok = ((idx >= 0) & (idx < E))[..., None]
    w = np.where(ok, gw[..., None].astype(np.float64), 0.0)
    o, do = o.reshape(T, k, -1), do.reshape(T, k, -1)
    y = (w * o).sum(axis=1)
    return y, (np.abs(w) * (do + 2 * U * (k + 1) * (np.abs(o) + do))).sum(axis=1)


@pytest.mark.parametrize("T, k, E, d, I, group", [
    (1, 1, 1, 32, 32, 32), (1, 8, 16, 256, 128, 128), (3, 2, 8, 256, 512, 64),
    (24, 1, 6, 128, 192, 64), (5, 3, 2, 96, 160, 32), (64, 8, 32, 128, 128, 128),
    (2, 8, 12, 7168, 256, 128), (1, 13, 40, 160, 96, 32),
])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ffn(T, k, E, d, I, group, dt):
    note(f"ffn T={T} k={k} E={E} d={d} I={I} group={group} {dt}")
    r = gen(T * 10 + k)
    w13, s13 = weights(r, E, 2 * I, d, group)
    w2, s2 = weights(r, E, d, I, group)
    idx = r.integers(0, E, (T, k)).astype(np.int32)
    gw = r.random((T, k)).astype(np.float32)
    if T * k > 2:
        idx[0, 0], gw[0, 0] = -1, np.nan             # a dropped slot's weight is not used
        idx[-1], gw[-1] = E, np.inf                  # a padding token
    x, x64 = rows(r, T, d, DT[dt])
    y, err = ffn_oracle(x64, OP.int4_weight(w13, s13), OP.int4_weight(w2, s2), idx, gw, d, I, group)
    args = (x, t_(w13), t_(s13), t_(w2), t_(s2), t_(idx), t_(gw))
    got = M.moe_ffn_int4(*args)
    check(got, y, err)
    if T * k > 2:
        assert torch.all(got[-1] == 0)
    ws = torch.full((M.moe_ffn_int4_workspace_size(T, k, d, I),), 255, dtype=torch.uint8,
                    device=dev())                    # whatever the workspace held before
    assert torch.equal(M.moe_ffn_int4(*args, workspace=ws), got)


@pytest.mark.parametrize("T, k, E, d, I, group", [
    # one token: 1, 2, 4 and 8 waves a slot, rounds of eight slots, ends of K inside a slice
    (1, 1, 3, 1056, 2080, 32), (1, 2, 9, 320, 1984, 64), (1, 3, 9, 128, 384, 128),
    (1, 4, 9, 224, 4128, 32), (1, 5, 9, 64, 64, 64), (1, 9, 12, 192, 896, 64),
    (1, 16, 16, 160, 32, 32), (1, 17, 20, 384, 1152, 128),
    # many slots an expert
    (96, 4, 3, 2080, 672, 32), (64, 4, 4, 1280, 1920, 64), (128, 8, 8, 1024, 640, 128),
    # many: gathered by expert
    (64, 8, 4, 256, 256, 64), (200, 2, 3, 224, 416, 32), (24, 1, 6, 1152, 640, 128),
    (2, 3, 5, 2080, 2080, 32),
])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ffn_of_one_token_and_of_many(T, k, E, d, I, group, dt):
    test_ffn(T, k, E, d, I, group, dt)


def test_ffn_of_one_token_without_an_expert():
    note("ffn one token, dropped")
    r = gen(77)
    w13, s13 = weights(r, 4, 128, 64, 32)
    w2, s2 = weights(r, 4, 64, 64, 32)
    idx = t_(np.array([[4, -1, 2 ** 31 - 1]], np.int32))
    x = torch.full((1, 64), float("nan"), device=dev())
    y = M.moe_ffn_int4(x, t_(w13), t_(s13), t_(w2), t_(s2), idx,
                       torch.full((1, 3), float("nan"), device=dev()))
    assert torch.all(y == 0)


@pytest.mark.parametrize("K, group", [(32, 32), (160, 32), (640, 128), (896, 128), (1088, 64)])
def test_matvec_scales_of_an_earlier_call_do_not_linger(K, group):
    """Blocks behind a row's end multiply zeros, whatever scales the shared memory still holds:
    here those of a call that left NaN and infinities in all of it."""
    note(f"matvec lingering scales K={K} group={group}")
    r = gen(K)
    q, s = weights(r, 1, 4096, 2048, 32)
    bad = np.full_like(s, np.nan)
    bad[:, ::2] = np.inf
    qk, sk = weights(r, 1, 300, K, group)
    x, x64 = rows(r, 1, K, torch.bfloat16)
    v, absum = OP.matvec_int4(x64, OP.int4_weight(qk, sk), None, 1)
    args = (x, t_(qk), t_(sk))
    first = (t_(np.zeros((1, 2048), np.float32), torch.bfloat16), t_(q), t_(bad))
    M.moe_matvec_int4(*first)
    y = M.moe_matvec_int4(*args)
    check(y, v, sum_error(absum, K, group))


# ---------------------------------------------------------------- balance loss

P_ERR = 2.0 ** -17   # fp32 softmax and sums: 12 u |key - max| + 28 u, then up to 67 additions


def router_case(r, T, E, k, spread=1.0):
    z = (r.standard_normal((T, E)) * spread + r.standard_normal((1, E)) * 0.5).astype(np.float32)
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    return z, idx


def check_balance(got, ref, kind, coef, E, n, live):
    loss, counts, probs, grad = (to_np(v).astype(np.float64) for v in got)
    rl, rc, rp, rg = ref
    np.testing.assert_array_equal(counts, rc)
    dP = P_ERR * rp
    assert np.all(np.abs(probs - rp) <= dP)
    each = np.where(n > 0, 1.0 / (np.maximum(n, 1) * max(live, 1)), 0.0)[:, None]
    if kind == "switch":
        # the oracle's own f - mean(f), f <= 1, is off by up to 2^-50 in fp64 (f's division, a sum
        # of E <= 1024 terms that add up to at most 1, and the mean's division: 2^-53 each); where
        # E counts_e is just the segment's sum of counts, 0 by the formula, that is all of it
        noise = 2.0 ** -50 * abs(coef) * E * each
        assert np.all(np.abs(grad - rg) <= 2 * U * np.abs(rg) + noise)
        tol = P_ERR * abs(rl)
    else:
        assert np.all(np.abs(grad - rg) <= abs(2 * coef) * each * dP + 2 * U * np.abs(rg))
        lv = (n > 0)[:, None]
        tol = abs(coef) * np.sum(lv * (2 * np.abs(rp - 1 / E) * dP + dP * dP)) / max(live, 1)
    assert abs(loss - rl) <= tol + 2 * U * abs(rl), (loss, rl, tol)


@pytest.mark.parametrize("T, E, k, B", [
    (1, 1, 1, 1), (1, 7, 2, 1), (5, 4, 4, 1), (63, 64, 6, 1), (130, 65, 3, 4), (257, 100, 8, 1),
    (1000, 256, 8, 7), (300, 520, 8, 3), (200, 1024, 64, 2), (4096, 33, 2, 1), (40, 16, 2, 60),
])
@pytest.mark.parametrize("kind", ["switch", "square"])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_loss(T, E, k, B, kind, masked):
    note(f"balance T={T} E={E} k={k} B={B} {kind} masked={masked}")
    r = gen(T + E)
    z, idx = router_case(r, T, E, k)
    idx[::7, 0] = [-1, E, 2 ** 31 - 1][T % 3]         # dropped slots are not counted
    bias = (r.random(E) * 0.02 - 0.01).astype(np.float32) if T % 2 else None
    mask = (r.random(T) < 0.8).astype(np.uint8) * 3 if masked else None
    off = None
    if B > 1:
        off = np.sort(r.integers(0, T + 1, B + 1)).astype(np.int32)
        off[2] = off[1]                              # an empty segment
    zz = z.copy()
    if masked:
        zz[mask == 0] = np.nan                       # what padding tokens hold has no influence
    ref = OP.balance_loss(z, idx, bias, mask, off, 0.37, kind)
    got = M.moe_balance_loss(t_(zz), t_(idx), None if bias is None else t_(bias),
                             None if mask is None else t_(mask), None if off is None else t_(off),
                             coef=0.37, kind=kind)
    segs = OP._counting(T, mask, off)
    n = np.array([len(s) for s in segs])
    check_balance(got, ref, kind, 0.37, E, n, int((n > 0).sum()))


@pytest.mark.parametrize("kind", ["switch", "square"])
def test_balance_without_tokens(kind):
    note(f"balance empty {kind}")
    z, idx = torch.empty((0, 8), device=dev()), torch.empty((0, 2), dtype=torch.int32, device=dev())
    off = torch.zeros(4, dtype=torch.int32, device=dev())
    for o, B in ((None, 1), (off, 3)):
        loss, counts, probs, grad = M.moe_balance_loss(z, idx, offsets=o, kind=kind)
        assert loss.item() == 0 and tuple(counts.shape) == (B, 8)
        assert not counts.any() and not probs.any() and not grad.any()
    z = torch.randn(5, 8, device=dev())
    loss, counts, probs, grad = M.moe_balance_loss(
        z, torch.zeros(5, 2, dtype=torch.int32, device=dev()),
        mask=torch.zeros(5, dtype=torch.bool, device=dev()), kind=kind)
    assert loss.item() == 0 and not counts.any() and not probs.any() and not grad.any()


def test_balance_masked_experts():
    """-inf and the type's lowest value as expert masks, a token with every expert masked, and
    NaN where it counts."""
    note("balance masked experts")
    r = gen(20)
    z, idx = router_case(r, 60, 70, 2)
    z[:, 5] = -np.inf
    z[3] = -np.inf
    z[4] = np.finfo(np.float32).min
    z[7, :60] = np.finfo(np.float32).min
    ref = OP.balance_loss(z, idx, kind="square", coef=1.0)
    got = M.moe_balance_loss(t_(z), t_(idx), kind="square", coef=1.0)
    check_balance(got, ref, "square", 1.0, 70, np.array([60]), 1)
    # expert 5 is masked for every token but number 4, whose 70 equal logits give it 1 / 70
    assert abs(got[2][0, 5].item() - 1 / (60 * 70)) <= P_ERR / (60 * 70)
    z[9, 9] = np.nan
    loss, counts, probs, grad = M.moe_balance_loss(t_(z), t_(idx), kind="square")
    assert torch.isnan(loss) and torch.isnan(probs).all() and torch.isnan(grad).all()
    np.testing.assert_array_equal(to_np(counts), ref[1])
    mask = torch.ones(60, dtype=torch.bool, device=dev())
    mask[9] = False
    assert torch.isfinite(M.moe_balance_loss(t_(z), t_(idx), mask=mask)[0])


def test_offsets_outside_the_batch_are_cut_to_it():
    """Offsets below 0 or past T name no token outside the batch."""
    note("offsets past T")
    r = gen(21)
    z, idx = router_case(r, 50, 9, 2)
    off = np.array([-3, 10, 30, 90], np.int32)
    ref = OP.balance_loss(z, idx, offsets=[0, 10, 30, 50], coef=1.0)
    got = M.moe_balance_loss(t_(z), t_(idx), offsets=t_(off), coef=1.0)
    check_balance(got, ref, "switch", 1.0, 9, np.array([10, 20, 20]), 3)
    g = r.standard_normal((3, 9)).astype(np.float32)
    a = M.moe_route_bwd(t_(z), offsets=t_(off), balance_grad=t_(g))
    b = M.moe_route_bwd(t_(z), offsets=t_(np.array([0, 10, 30, 50], np.int32)), balance_grad=t_(g))
    assert torch.equal(a, b)


@pytest.mark.parametrize("T, E, k, B", [
    # several turns of tokens a part; more segments than one part each, and two parts each
    (40000, 48, 2, 1), (33000, 100, 3, 5), (20000, 512, 2, 1), (3000, 9, 2, 700), (3000, 9, 2, 400),
    (9000, 300, 40, 1),
])
def test_balance_loss_of_larger_batches(T, E, k, B):
    test_balance_loss(T, E, k, B, "switch", True)
    test_balance_loss(T, E, k, B, "square", False)


# ------------------------------------------------------------- router backward

@pytest.mark.parametrize("T, E, k, B", [
    (1, 1, 1, 1), (1, 5, 2, 1), (3, 64, 6, 1), (77, 65, 3, 4), (257, 256, 8, 1), (500, 256, 8, 9),
    (90, 300, 7, 2), (60, 1024, 64, 1), (5000, 16, 2, 1), (40, 16, 2, 60), (9, 2, 2, 1),
])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("parts", ["gate", "balance", "both"])
def test_route_bwd(T, E, k, B, renorm, parts):
    note(f"route bwd T={T} E={E} k={k} B={B} renorm={renorm} {parts}")
    r = gen(T * 3 + E)
    z, idx = router_case(r, T, E, k)
    idx[::7, 0] = [-1, E, -2 ** 31][T % 3]
    if k > 1:
        idx[1::5, 1] = idx[1::5, 0]                  # an expert twice
    bias = (r.random(E) * 0.02 - 0.01).astype(np.float32) if T % 2 else None
    mask = (r.random(T) < 0.8).astype(np.uint8) if T % 3 else None
    off = np.sort(r.integers(0, T + 1, B + 1)).astype(np.int32) if B > 1 else None
    dw = r.standard_normal((T, k)).astype(np.float32) if parts != "balance" else None
    g = r.standard_normal((B, E)).astype(np.float32) if parts != "gate" else None
    dloss = np.float32(1.7)
    ref, mag = OP.route_bwd(z, idx, dw, bias, renorm, mask, off, g, dloss)
    zz, dd = z.copy(), None if dw is None else dw.copy()
    counted = np.zeros(T, bool)
    for s in OP._counting(T, mask, off):
        counted[s] = True
    zz[~counted] = np.nan                            # rows that do not count
    if dd is not None:
        dd[~counted] = np.nan
        dd[(idx < 0) | (idx >= E)] = np.inf          # slots without an expert
    o = lambda v: None if v is None else t_(v)  # noqa: E731
    call = dict(dtopk_w=o(dd), bias=o(bias), renorm=renorm, mask=o(mask), offsets=o(off),
                balance_grad=o(g), dloss=t_(np.array([dloss])) if g is not None else None)
    dz, db = M.moe_route_bwd(t_(zz), t_(idx), need_dbias=True, **call)
    tol = P_ERR * mag + 2 * U * np.abs(ref)
    assert np.all(np.abs(to_np(dz) - ref) <= tol)
    assert not dz[t_(~counted)].any()
    # dbias: at most T / 4 + 3 fp32 additions in a row, then fp64
    chain = 2 * U * (T // 4 + 4)
    assert np.all(np.abs(to_np(db) - ref.sum(axis=0)) <=
                  tol.sum(axis=0) + chain * (np.abs(ref) + tol).sum(axis=0))
    assert torch.equal(M.moe_route_bwd(t_(zz), t_(idx), **call), dz)


@pytest.mark.parametrize("T, E, k, B", [
    # more slots than a token has lanes
    (20, 64, 9, 1), (33, 100, 20, 2), (50, 200, 33, 1), (21, 400, 40, 1),
    # several turns of tokens a workgroup
    (40000, 20, 3, 3), (36000, 120, 2, 1), (20000, 130, 17, 6),
])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_bwd_of_larger_batches(T, E, k, B, renorm):
    test_route_bwd(T, E, k, B, renorm, "both")


def test_route_bwd_masked_experts():
    note("route bwd masked experts")
    r = gen(30)
    z, idx = router_case(r, 40, 70, 3)
    z[:, 6] = -np.inf
    z[3] = -np.inf
    z[4] = np.finfo(np.float32).min
    dw = r.standard_normal((40, 3)).astype(np.float32)
    g = r.standard_normal((1, 70)).astype(np.float32)
    for renorm in (False, True):
        ref, mag = OP.route_bwd(z, idx, dw, renorm=renorm, balance_grad=g)
        dz = M.moe_route_bwd(t_(z), t_(idx), dtopk_w=t_(dw), renorm=renorm, balance_grad=t_(g))
        assert np.all(np.abs(to_np(dz) - ref) <= P_ERR * mag + 2 * U * np.abs(ref))
        masked = torch.arange(40, device=dev()) != 4       # row 4's logits are all equal
        assert not dz[3].any() and not dz[masked, 6].any()


def test_route_bwd_without_tokens():
    note("route bwd empty")
    z, idx = torch.empty((0, 8), device=dev()), torch.empty((0, 2), dtype=torch.int32, device=dev())
    dz, db = M.moe_route_bwd(z, idx, dtopk_w=torch.empty((0, 2), device=dev()), need_dbias=True)
    assert dz.numel() == 0 and not db.any()


@pytest.mark.parametrize("kind", ["switch", "square"])
def test_gradient_against_differences_of_the_loss(kind):
    """The loss along the direction d = sign(dlogits): (L(z + h d) - L(z - h d)) / 2h against
    sum |dlogits|.  P moves by at most 2 h P, so the quotient's truncation is at most
    (2h)^2 of the loss's own terms; the loss's rounding (2^-17 of its terms at most, and in
    fact their mean over T tokens) is divided by 2 h."""
    note(f"differences {kind}")
    r = gen(40)
    T, E, k, h = 512, 16, 2, 2.0 ** -5
    z, idx = router_case(r, T, E, k)
    z = (np.round(z * 256) / 256).astype(np.float32)
    loss, _, _, g = M.moe_balance_loss(t_(z), t_(idx), coef=1.0, kind=kind)
    dz = to_np(M.moe_route_bwd(t_(z), t_(idx), balance_grad=g)).astype(np.float64)
    d = np.where(dz >= 0, 1.0, -1.0).astype(np.float32)
    up, down = (M.moe_balance_loss(t_(z + s * h * d), t_(idx), coef=1.0, kind=kind)[0].item()
                for s in (1, -1))
    terms = 1.0 if kind == "switch" else 2.0
    tol = terms * (4 * h * h * np.abs(dz).sum() * 4 + 2.0 ** -17 / (2 * h) * loss.item())
    assert abs((up - down) / (2 * h) - np.abs(dz).sum()) <= tol


# ------------------------------------------------------- together, and as used

def test_training_step_of_the_router():
    """moe_route, moe_balance_loss and moe_route_bwd as a training step uses them: the loss
    and the gradient are those of the oracle on the kernel's own logits, and the counts are
    the dispatch's."""
    note("router training step")
    r = gen(50)
    T, d, E, k = 300, 512, 64, 6
    x = t_(r.standard_normal((T, d)).astype(np.float32), torch.bfloat16)
    w = t_((r.standard_normal((E, d)) * d ** -0.5).astype(np.float32), torch.bfloat16)
    bias = t_((r.random(E) * 0.02 - 0.01).astype(np.float32))
    off = t_(np.array([0, 100, 100, 290], np.int32))
    for renorm in (False, True):
        idx, gw, logits = M.moe_route(x, w, bias, k, renorm=renorm)
        loss, counts, probs, grad = M.moe_balance_loss(logits, idx, bias=bias, coef=0.1)
        assert torch.equal(counts[0], M.moe_dispatch(idx, E, 16)[0])
        dw = t_(r.standard_normal((T, k)).astype(np.float32))
        dz, db = M.moe_route_bwd(logits, idx, dtopk_w=dw, bias=bias, renorm=renorm,
                                 balance_grad=grad, need_dbias=True)
        z, i, b = to_np(logits), to_np(idx), to_np(bias)
        check_balance((loss, counts, probs, grad), OP.balance_loss(z, i, b, coef=0.1), "switch",
                      0.1, E, np.array([T]), 1)
        wo, _, _ = OP.gate_weights(z, i, b, renorm)
        assert np.all(np.abs(to_np(gw) - wo) <= 2.0 ** -17 * wo)
        ref, mag = OP.route_bwd(z, i, to_np(dw), b, renorm, balance_grad=to_np(grad))
        assert np.all(np.abs(to_np(dz) - ref) <= P_ERR * mag + 2 * U * np.abs(ref))
        # the sequence-wise loss of the same routing leaves the last 10 tokens out
        _, seq, _, g2 = M.moe_balance_loss(logits, idx, bias=bias, offsets=off)
        assert int(seq.sum()) == 290 * k
        dz2 = M.moe_route_bwd(logits, bias=bias, offsets=off, balance_grad=g2)
        assert not dz2[290:].any() and dz2[:290].any()


@pytest.mark.parametrize("T", [1, 5])
def test_decode_step_against_the_layer(T):
    """moe_route and moe_ffn_int4 against moe_layer_fwd with the same int4 weights: the layer
    rounds the weights to bf16 (2^-9 of each product), h and each expert row to bf16."""
    note(f"decode step T={T}")
    r = gen(60 + T)
    d, E, k, I = 512, 16, 4, 256
    x = t_(r.standard_normal((T, d)).astype(np.float32), torch.bfloat16)
    wr = t_((r.standard_normal((E, d)) * d ** -0.5).astype(np.float32), torch.bfloat16)
    bias = t_((r.random(E) * 0.02).astype(np.float32))
    w13, s13 = M.moe_quant_weight_int4(t_((r.standard_normal((E, 2 * I, d)) * d ** -0.5)
                                          .astype(np.float32)))
    w2, s2 = M.moe_quant_weight_int4(t_((r.standard_normal((E, d, I)) * I ** -0.5)
                                        .astype(np.float32)))
    desc = M.LayerDesc(T, d, E, k, I, mode="w4a16", m_align=16)
    y0, _ = M.moe_layer_fwd(desc, {"w_router": wr, "bias": bias, "w13": w13, "s13": s13, "w2": w2,
                                   "s2": s2}, x)
    idx, gw, _ = M.moe_route(x, wr, bias, k)
    y1 = M.moe_ffn_int4(x, w13, s13, w2, s2, idx, gw)
    a, b = to_np(y0).astype(np.float64), to_np(y1).astype(np.float64)
    # root mean square: two weight roundings, h, o and the two y's, each uniform in +-2^-9
    # relative to its terms (standard deviation 2^-9/sqrt(3)), silu's slope at most 1.1
    rms = np.sqrt(np.mean((a - b) ** 2)) / np.sqrt(np.mean(b ** 2))
    assert rms <= 3 * 2.0 ** -9 * np.sqrt(6 / 3), rms


def _ops(seed):
    """One call of each operator on fixed inputs, as a function of nothing."""
    r = gen(seed)
    T, k, E, d, I = 6, 4, 16, 256, 128
    w13, s13 = (t_(v) for v in weights(r, E, 2 * I, d, 64))
    w2, s2 = (t_(v) for v in weights(r, E, d, I, 64))
    x, _ = rows(r, T, d, torch.bfloat16)
    z, idx = router_case(r, 500, E, k)
    zt, it = t_(z), t_(idx)
    gw = t_(r.random((T, k)).astype(np.float32))
    off = t_(np.array([0, 200, 460], np.int32))
    dw = t_(r.standard_normal((500, k)).astype(np.float32))
    fi = it[:T].contiguous()

    def call():
        y = M.moe_ffn_int4(x, w13, s13, w2, s2, fi, gw)
        v = M.moe_matvec_int4(x, w13, s13, fi.view(-1), x_div=k, swiglu=True)
        loss, c, p, g = M.moe_balance_loss(zt, it, offsets=off, coef=1.0)
        dz, db = M.moe_route_bwd(zt, it, dtopk_w=dw, offsets=off, balance_grad=g, need_dbias=True)
        return [y, v, loss, c, p, g, dz, db]
    return call, x


def test_repeatable_and_on_any_stream():
    note("repeat, streams")
    call, _ = _ops(70)
    want = [v.clone() for v in call()]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in side * 2:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(call())
    torch.cuda.synchronize()
    for one in got:
        for a, b in zip(one, want):
            assert torch.equal(a, b)


def test_gathered_calls_on_streams_and_captured():
    """The same for the calls that take the other variants: an FFN gathered by expert, a loss
    joined from many parts, more slots than lanes; two streams at once, and a graph replayed
    among eager calls."""
    note("gathered, streams and graph")
    r = gen(72)
    T, k, E, d, I = 64, 8, 4, 1024, 256
    w13, s13 = (t_(v) for v in weights(r, E, 2 * I, d, 64))
    w2, s2 = (t_(v) for v in weights(r, E, d, I, 64))
    x, _ = rows(r, T, d, torch.bfloat16)
    fi = t_(r.integers(-1, E, (T, k)).astype(np.int32))
    gw = t_(r.random((T, k)).astype(np.float32))
    z, idx = router_case(r, 20000, 64, 12)
    zt, it = t_(z), t_(idx)
    dw = t_(r.standard_normal((20000, 12)).astype(np.float32))

    def call():
        y = M.moe_ffn_int4(x, w13, s13, w2, s2, fi, gw)
        loss, c, p, g = M.moe_balance_loss(zt, it, coef=1.0, kind="square")
        dz, db = M.moe_route_bwd(zt, it, dtopk_w=dw, renorm=True, balance_grad=g, dloss=loss,
                                 need_dbias=True)
        return [y, loss, c, p, g, dz, db]

    want = [v.clone() for v in call()]
    got = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(call())
    torch.cuda.synchronize()
    for one in got:
        for a, b in zip(one, want):
            assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for i in range(4):
        x.copy_(torch.randn_like(x, dtype=torch.float32).to(x.dtype))
        zt.copy_(torch.randn_like(zt))
        want = [v.clone() for v in call()]
        for v in out:
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i


def test_captured_and_replayed():
    """A captured graph gives the eager results on every replay, with eager calls between the
    replays and inputs changed in place."""
    note("graph")
    call, x = _ops(71)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for i in range(4):
        x.copy_(torch.randn_like(x, dtype=torch.float32).to(x.dtype))
        want = [v.clone() for v in call()]
        for v in out:
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i
