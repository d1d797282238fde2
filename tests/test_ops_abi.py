"""Host-side checks of the operators of include/moe_ops.h: every symbol is exported and
bound, and bad arguments are refused before a device is touched.  No kernel runs here."""
import ctypes as C
import os
import re

import pytest
import torch

import fp8_grouped_gemm_amd as M
from fp8_grouped_gemm_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = C.c_void_p(0x1000)   # never dereferenced: validation rejects the call first
ODD = C.c_void_p(0x1002)
BF16, F32 = _lib.MOE_BF16, _lib.MOE_F32


def test_header_symbols_exported():
    src = open(os.path.join(ROOT, "include", "moe_ops.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    declared = re.findall(r"^\s*(?:int|size_t)\s+([a-z_0-9]+)\s*\(", src, flags=re.M)
    assert sorted(declared) == sorted(_lib.SIGNATURES_OPS)
    for name in declared:
        assert hasattr(_lib.load(), name), name
    assert int(re.search(r"MOE_FEW_SLOTS_MAX (\d+)", src).group(1)) == _lib.MOE_FEW_SLOTS_MAX


def _err(status, fragment, code=_lib.MOE_ERR_INVALID_ARG):
    assert status == code
    msg = _lib.load().moe_last_error().decode()
    assert fragment in msg, msg


def _matvec(x=FAKE, x_dt=BF16, x_div=1, q=FAKE, s7=FAKE, group=128, idx=FAKE, S=4, G=8, N=16,
            K=256, epi=0, y=FAKE, y_dt=BF16):
    return _lib.load().moe_matvec_int4(x, x_dt, x_div, q, s7, group, idx, S, G, N, K, epi, y, y_dt,
                                       None)


@pytest.mark.parametrize("kw, fragment", [
    ({"x": None}, "null"), ({"q": None}, "null"), ({"s7": None}, "null"), ({"y": None}, "null"),
    ({"x_dt": _lib.MOE_E4M3}, "dtypes"), ({"y_dt": _lib.MOE_INT4}, "dtypes"),
    ({"group": 16}, "group must"), ({"group": 0}, "group must"), ({"group": 256}, "group must"),
    ({"K": 192}, "multiple of group"), ({"K": 0}, "multiple of group"),
    ({"K": -128}, "multiple of group"), ({"N": 0}, "N must"), ({"N": (1 << 24) + 1}, "N must"),
    ({"G": 0}, "G must"), ({"S": -1}, "S must"), ({"S": 1025}, "grouped GEMMs"),
    ({"x_div": 0}, "x_div"), ({"epi": 2}, "epilogue"), ({"x": ODD}, "aligned"),
    ({"q": ODD}, "aligned"), ({"idx": None, "x_div": 2}, "x_div"), ({"K": 1 << 25}, "K must"),
])
def test_matvec_refuses(kw, fragment):
    _err(_matvec(**kw), fragment)


def test_no_slots_is_no_work():
    assert _matvec(S=0, x=None, y=None, idx=None) == _lib.MOE_OK


def _ffn(x=FAKE, dt=BF16, w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE, group=128, idx=FAKE, w=FAKE, T=2,
         k=2, E=4, d=256, I=128, y=FAKE, ws=FAKE, n=1 << 30):
    return _lib.load().moe_ffn_int4(x, dt, w13, s13, w2, s2, group, idx, w, T, k, E, d, I, y, ws, n,
                                    None)


@pytest.mark.parametrize("kw, fragment", [
    ({"x": None}, "null"), ({"w2": None}, "null"), ({"idx": None}, "null"), ({"w": None}, "null"),
    ({"ws": None}, "null"), ({"dt": _lib.MOE_E4M3}, "dt must"), ({"group": 48}, "group must"),
    ({"d": 200}, "multiples of group"), ({"I": 0}, "multiples of group"), ({"E": 0}, "E must"),
    ({"T": -1}, "T >= 0"), ({"k": 0}, "T * k"), ({"T": 600}, "moe_layer_fwd"),
    ({"T": 1 << 30, "k": 4}, "T * k"), ({"ws": ODD}, "aligned"), ({"w13": ODD}, "aligned"),
    ({"d": 1 << 25}, "2^24"),
])
def test_ffn_refuses(kw, fragment):
    _err(_ffn(**kw), fragment)


def test_ffn_workspace():
    lib = _lib.load()
    assert lib.moe_ffn_int4_workspace_size(4, 2, 256, 128) >= 8 * 128 * 4
    assert lib.moe_ffn_int4_workspace_size(600, 2, 256, 128) == 0
    assert lib.moe_ffn_int4_workspace_size(0, 2, 256, 128) == 0
    _err(_ffn(n=16), "workspace", _lib.MOE_ERR_WORKSPACE)
    assert _ffn(T=0, x=None, y=None, idx=None, w=None, ws=None, n=0) == _lib.MOE_OK


def test_quant_group_refuses():
    lib = _lib.load()
    _err(lib.moe_quant_weight_int4_group(None, 1, 4, 64, 64, FAKE, FAKE, None), "null")
    _err(lib.moe_quant_weight_int4_group(FAKE, 1, 4, 64, 16, FAKE, FAKE, None), "group must")
    _err(lib.moe_quant_weight_int4_group(FAKE, 1, 4, 96, 64, FAKE, FAKE, None), "multiple of group")
    _err(lib.moe_quant_weight_int4_group(FAKE, 0, 4, 64, 64, FAKE, FAKE, None), "bad G/N")
    _err(lib.moe_quant_weight_int4_group(ODD, 1, 4, 64, 64, FAKE, FAKE, None), "aligned")
    big = 1 << 30
    _err(lib.moe_quant_weight_int4_group(FAKE, big, big, 64, 64, FAKE, FAKE, None), "too large")


def _balance(logits=FAKE, bias=None, idx=FAKE, mask=None, off=None, T=8, E=16, k=2, B=1, kind=0,
             coef=0.01, counts=FAKE, probs=FAKE, grad=FAKE, loss=FAKE, ws=FAKE, n=1 << 30):
    return _lib.load().moe_balance_loss(logits, bias, idx, mask, off, T, E, k, B, kind, coef,
                                        counts, probs, grad, loss, ws, n, None)


@pytest.mark.parametrize("kw, fragment", [
    ({"logits": None}, "null"), ({"idx": None}, "null"), ({"loss": None}, "null"),
    ({"ws": None}, "null"), ({"counts": None}, "null"), ({"T": -1}, "T must"),
    ({"E": 0}, "E must"), ({"E": 1025}, "E must"), ({"k": 0}, "k must"), ({"k": 17}, "k must"),
    ({"E": 128, "k": 65}, "k must"), ({"B": 0}, "B must"), ({"B": 65536, "off": FAKE}, "B must"),
    ({"B": 2}, "offsets"), ({"kind": 2}, "kind"), ({"coef": float("nan")}, "finite"),
    ({"coef": float("inf")}, "finite"), ({"ws": ODD}, "aligned"),
])
def test_balance_refuses(kw, fragment):
    _err(_balance(**kw), fragment)


def test_balance_workspace():
    lib = _lib.load()
    assert lib.moe_balance_workspace_size(8, 16, 1) > 0
    assert lib.moe_balance_workspace_size(0, 16, 1) > 0
    assert lib.moe_balance_workspace_size(-1, 16, 1) == 0
    assert lib.moe_balance_workspace_size(8, 2000, 1) == 0
    _err(_balance(n=16), "workspace", _lib.MOE_ERR_WORKSPACE)


def _bwd(logits=FAKE, bias=None, idx=FAKE, dw=FAKE, mask=None, off=None, grad=None, dloss=None,
         T=8, E=16, k=2, B=1, flags=0, dlogits=FAKE, dbias=None, ws=None, n=0):
    return _lib.load().moe_route_bwd(logits, bias, idx, dw, mask, off, grad, dloss, T, E, k, B,
                                     flags, dlogits, dbias, ws, n, None)


@pytest.mark.parametrize("kw, fragment", [
    ({"logits": None}, "null"), ({"dlogits": None}, "null"), ({"dw": None}, "is needed"),
    ({"idx": None}, "topk_idx"), ({"flags": 2}, "flags"), ({"T": -1}, "T must"),
    ({"E": 4096}, "E must"), ({"k": 17}, "k must"), ({"B": 3}, "offsets"),
    ({"dbias": FAKE}, "workspace"), ({"dbias": FAKE, "ws": ODD, "n": 1 << 20}, "aligned"),
])
def test_route_bwd_refuses(kw, fragment):
    _err(_bwd(**kw), fragment)


def test_route_bwd_workspace():
    assert _lib.load().moe_route_bwd_workspace_size(8, 16) > 0
    assert _lib.load().moe_route_bwd_workspace_size(8, 0) == 0
    _err(_bwd(dbias=FAKE, ws=FAKE, n=16), "workspace", _lib.MOE_ERR_WORKSPACE)
    assert _bwd(T=0, logits=None, dlogits=None, idx=None) == _lib.MOE_OK


def test_binding_refuses_wrong_tensors():
    """Shapes and dtypes are refused by the binding before the library is called (CPU
    tensors here: a call that passed these checks would be refused as not on the GPU)."""
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    q, s = torch.zeros(4, 32, 64, dtype=u8), torch.ones(4, 32, 1)
    x = torch.zeros(2, 128)
    idx = torch.zeros(2, dtype=i32)
    bad = [
        lambda: M.moe_matvec_int4(x, q.to(torch.int8), s, idx),
        lambda: M.moe_matvec_int4(x, q, s[:2], idx),
        lambda: M.moe_matvec_int4(x, q, s.half(), idx),
        lambda: M.moe_matvec_int4(x, q, s, idx.long()),
        lambda: M.moe_matvec_int4(x, q, s, idx, x_div=2),
        lambda: M.moe_matvec_int4(x, q, s, idx, x_div=0),
        lambda: M.moe_matvec_int4(x, q, s, x_div=2),
        lambda: M.moe_matvec_int4(x[:, :64], q, s, idx),
        lambda: M.moe_matvec_int4(x, q[:, :31], s[:, :31], idx, swiglu=True),
        lambda: M.moe_matvec_int4(x.half(), q, s, idx),
        lambda: M.moe_quant_weight_int4_group(torch.zeros(1, 4, 96), 64),
        lambda: M.moe_quant_weight_int4_group(torch.zeros(1, 4, 96, dtype=torch.bfloat16), 32),
    ]
    w2, s2 = torch.zeros(4, 128, 8, dtype=u8), torch.ones(4, 128, 1)
    k2 = torch.zeros(2, 3, dtype=i32)
    w = torch.zeros(2, 3)
    bad += [
        lambda: M.moe_ffn_int4(x, q, s, w2, s2, k2, w),          # group 128 and 16
        lambda: M.moe_ffn_int4(x, q, s, q, s, k2, w),
    ]
    z = torch.zeros(5, 8)
    at = torch.zeros(5, 2, dtype=i32)
    bad += [
        lambda: M.moe_balance_loss(z.double(), at),
        lambda: M.moe_balance_loss(z, at.long()),
        lambda: M.moe_balance_loss(z, at[:4]),
        lambda: M.moe_balance_loss(z, at, bias=torch.zeros(7)),
        lambda: M.moe_balance_loss(z, at, mask=torch.ones(5)),
        lambda: M.moe_balance_loss(z, at, offsets=torch.zeros(3)),
        lambda: M.moe_balance_loss(z, at, kind="cv"),
        lambda: M.moe_route_bwd(z, at, dtopk_w=torch.zeros(5, 3)),
        lambda: M.moe_route_bwd(z, at, dtopk_w=torch.zeros(5, 2), balance_grad=torch.zeros(2, 8)),
        lambda: M.moe_route_bwd(z, at, dtopk_w=torch.zeros(5, 2), dloss=torch.zeros(2)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError) as e:
            call()
        assert "on the GPU" not in str(e.value), (i, str(e.value))
    with pytest.raises(ValueError, match="on the GPU"):
        M.moe_balance_loss(z, at)
