"""MI355X (gfx950) forward pass of one Mixture-of-Experts FFN layer.

A thin binding over the C ABI of ``libmoe_gfx950.so`` (include/moe.h, and
include/moe_ops.h for the operators beside the layer forward): each function here
has the C entry point's name, takes torch tensors that live on the GPU, allocates
the outputs with torch and passes raw pointers plus the current HIP stream.  Every
step runs in the library's HIP kernels; nothing is computed in Python.
"""
from __future__ import annotations

import ctypes as C
import functools
from typing import Optional

import torch

from . import _lib
from ._lib import (MOE_BF16, MOE_E4M3, MOE_EPI_PLAIN, MOE_EPI_SWIGLU, MOE_F32, MOE_INT4,
                   MOE_MODE_FP32, MOE_MODE_FP8, MOE_MODE_W4A16, MOE_MODE_W4A8, MOE_ROUTE_HASH,
                   MOE_ROUTE_RENORM, MOE_ROUTE_SCORE, MoeError, MoeLayerDesc, MoeLayerWeights)

__all__ = [
    "moe_device_supported", "moe_capacity", "moe_rows_bound", "moe_route", "moe_route_noalloc",
    "moe_route_from_logits", "moe_route_hash", "moe_route_workspace_size", "moe_dispatch",
    "moe_dispatch_masked", "moe_quant_fp8",
    "moe_quant_weight_fp8", "moe_pack_weight_fp8", "moe_quant_weight_int4", "moe_pack_weight_int4",
    "grouped_gemm_fp8", "grouped_gemm_fp8_masked", "grouped_gemm_w4a8",
    "gemm_fp8", "grouped_gemm_w4a16",
    "grouped_gemm_f32", "moe_combine", "moe_layer_workspace_size", "moe_layer_fwd", "MoeError",
    "moe_layer_chunked_workspace_size", "moe_layer_fwd_chunked",
    "LayerDesc", "moe_probe_mfma_fp8", "moe_probe_hbm_read",
    "moe_quant_weight_int4_group", "moe_matvec_int4", "moe_ffn_int4", "moe_balance_loss",
    "moe_route_bwd",
]


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(dev: torch.device):
    """The handle of torch's current stream on dev (without the Stream object around it)."""
    i = dev.index if dev.index is not None else torch.cuda.current_device()
    return torch._C._cuda_getCurrentRawStream(i)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


def _lib_():
    return _lib.load()


def _on_tensor_device(fn):
    """Run fn with the device of its GPU tensor arguments (and of the tensors in a dict
    argument, such as the layer's weights) current.  The library checks and launches on
    the current HIP device, and the stream passed in belongs to the tensors' device, so
    the two must agree; tensors on different GPUs are refused."""
    @functools.wraps(fn)
    def call(*args, **kwargs):
        index = -1
        for a in (*args, *kwargs.values()):
            if isinstance(a, torch.Tensor):
                i = a.get_device()                  # -1 for a host tensor
                if i != index and i >= 0:
                    if index >= 0:
                        refuse(index, i)
                    index = i
            elif isinstance(a, dict):
                for t in a.values():
                    if isinstance(t, torch.Tensor) and t.is_cuda:
                        if index >= 0 and t.get_device() != index:
                            refuse(index, t.get_device())
                        index = t.get_device()
        if index < 0 or index == torch._C._cuda_getDevice():
            return fn(*args, **kwargs)
        with torch.cuda.device(index):
            return fn(*args, **kwargs)

    def refuse(*indices):
        raise ValueError(f"{fn.__name__}: tensors on different devices "
                         f"{sorted(f'cuda:{i}' for i in indices)}")
    return call


# --------------------------------------------------------------- host helpers

def moe_device_supported(device: int = 0) -> bool:
    return _lib_().moe_device_supported(device) == _lib.MOE_OK


def moe_capacity(T: int, k: int, E: int, factor: float) -> int:
    r = _lib_().moe_capacity(T, k, E, float(factor))
    _lib.check(min(r, 0), "moe_capacity")
    return r


def moe_rows_bound(T: int, k: int, E: int, m_align: int) -> int:
    return _lib_().moe_rows_bound(T, k, E, m_align)


# -------------------------------------------------------------------- routing

@_on_tensor_device
def moe_route(x: torch.Tensor, w_router: torch.Tensor, bias: torch.Tensor, k: int,
              renorm: bool = False, use_workspace: bool = True):
    """Router logits + biased softmax top-k.  Returns (topk_idx, topk_w, logits).
    use_workspace=False passes no workspace (the logits GEMM then runs without split-K)."""
    T, d = x.shape
    E = w_router.shape[0]
    dev = x.device
    logits = torch.empty((T, E), dtype=torch.float32, device=dev)
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    nws = _lib_().moe_route_workspace_size(T, d, E, _dt(x)) if use_workspace else 0
    ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=dev)
    _lib.check(_lib_().moe_route(_ptr(x), _dt(x), _ptr(w_router), _ptr(bias), T, d, E, k,
                                 MOE_ROUTE_RENORM if renorm else 0, _ptr(logits), _ptr(idx),
                                 _ptr(w), _ptr(ws), nws, _stream(dev)), "moe_route")
    return idx, w, logits


@_on_tensor_device
def moe_route_noalloc(x: torch.Tensor, w_router: torch.Tensor, bias: torch.Tensor, k: int,
                      renorm: bool = False, out=None):
    """moe_route with the split-K partials in the library's static device scratch (no
    device allocation inside the call).  ``out`` = (topk_idx, topk_w, logits) tensors to
    write, or None to allocate them here with torch.  Returns (topk_idx, topk_w, logits)."""
    T, d = x.shape
    E = w_router.shape[0]
    dev = x.device
    if out is None:
        out = (torch.empty((T, k), dtype=torch.int32, device=dev),
               torch.empty((T, k), dtype=torch.float32, device=dev),
               torch.empty((T, E), dtype=torch.float32, device=dev))
    idx, w, logits = out
    _lib.check(_lib_().moe_route_noalloc(_ptr(x), _dt(x), _ptr(w_router), _ptr(bias), T, d, E,
                                         k, MOE_ROUTE_RENORM if renorm else 0, _ptr(logits),
                                         _ptr(idx), _ptr(w), _stream(dev)), "moe_route_noalloc")
    return idx, w, logits


def moe_route_workspace_size(T: int, d: int, E: int, dtype=torch.bfloat16) -> int:
    return _lib_().moe_route_workspace_size(T, d, E, MOE_BF16 if dtype == torch.bfloat16 else MOE_F32)


@_on_tensor_device
def moe_route_from_logits(logits: torch.Tensor, bias: Optional[torch.Tensor], k: int,
                          renorm: bool = False):
    T, E = logits.shape
    dev = logits.device
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    _lib.check(_lib_().moe_route_from_logits(_ptr(logits), _ptr(bias), T, E, k,
                                             MOE_ROUTE_RENORM if renorm else 0, _ptr(idx),
                                             _ptr(w), _stream(dev)), "moe_route_from_logits")
    return idx, w


@_on_tensor_device
def moe_route_hash(token_ids: torch.Tensor, E: int):
    T = token_ids.shape[0]
    dev = token_ids.device
    idx = torch.empty((T, 1), dtype=torch.int32, device=dev)
    w = torch.empty((T, 1), dtype=torch.float32, device=dev)
    _lib.check(_lib_().moe_route_hash(_ptr(token_ids), T, E, _ptr(idx), _ptr(w), _stream(dev)),
               "moe_route_hash")
    return idx, w


@_on_tensor_device
def moe_dispatch(topk_idx: torch.Tensor, E: int, m_align: int, capacity: int = 0):
    """Returns (counts [E], offsets [E+1], row_of_slot [T*k], slot_of_row [rows_bound])."""
    T, k = topk_idx.shape
    dev = topk_idx.device
    R = moe_rows_bound(T, k, E, m_align)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    ros = torch.empty(T * k, dtype=torch.int32, device=dev)
    sor = torch.empty(R, dtype=torch.int32, device=dev)
    _lib.check(_lib_().moe_dispatch(_ptr(topk_idx), T, k, E, m_align, capacity, _ptr(counts),
                                    _ptr(offsets), _ptr(ros), _ptr(sor), _stream(dev)),
               "moe_dispatch")
    return counts, offsets, ros, sor


@_on_tensor_device
def moe_dispatch_masked(topk_idx: torch.Tensor, E: int, capacity: int):
    """Fixed-capacity layout.  Returns (counts [E], row_of_slot [T*k], slot_of_row [E*C])."""
    T, k = topk_idx.shape
    dev = topk_idx.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    ros = torch.empty(T * k, dtype=torch.int32, device=dev)
    sor = torch.empty(E * capacity, dtype=torch.int32, device=dev)
    _lib.check(_lib_().moe_dispatch_masked(_ptr(topk_idx), T, k, E, capacity, _ptr(counts),
                                           _ptr(ros), _ptr(sor), _stream(dev)),
               "moe_dispatch_masked")
    return counts, ros, sor


# --------------------------------------------------------------- quantisation

@_on_tensor_device
def moe_quant_fp8(x: torch.Tensor, src_row: Optional[torch.Tensor] = None, src_div: int = 1,
                  rows_out: Optional[int] = None):
    """1x128 e4m3 quantisation; returns (codes uint8 [rows_out, K], scales fp32)."""
    rows_in, K = x.shape
    rows_out = rows_in if rows_out is None else rows_out
    dev = x.device
    q = torch.empty((rows_out, K), dtype=torch.uint8, device=dev)
    s = torch.empty((rows_out, K // 128), dtype=torch.float32, device=dev)
    _lib.check(_lib_().moe_quant_fp8(_ptr(x), _dt(x), rows_in, K, _ptr(src_row), src_div,
                                     rows_out, _ptr(q), _ptr(s), _stream(dev)), "moe_quant_fp8")
    return q, s


@_on_tensor_device
def moe_quant_weight_fp8(w: torch.Tensor):
    G, N, K = w.shape
    dev = w.device
    q = torch.empty((G, N, K), dtype=torch.uint8, device=dev)
    s = torch.empty((G, N // 128, K // 128), dtype=torch.float32, device=dev)
    _lib.check(_lib_().moe_quant_weight_fp8(_ptr(w), G, N, K, _ptr(q), _ptr(s), _stream(dev)),
               "moe_quant_weight_fp8")
    return q, s


@_on_tensor_device
def moe_pack_weight_fp8(q: torch.Tensor):
    """e4m3 codes [G, N, K] (or [N, K]) -> the fragment-major layout the FP8 GEMMs read
    (same shape and byte count; see moe_pack_weight_fp8 in include/moe.h)."""
    q3 = q if q.dim() == 3 else q[None]
    G, N, K = q3.shape
    q3 = q3.contiguous()                  # kept alive until the launch is enqueued
    out = torch.empty_like(q3)
    _lib.check(_lib_().moe_pack_weight_fp8(_ptr(q3), G, N, K, _ptr(out), _stream(q.device)),
               "moe_pack_weight_fp8")
    return out if q.dim() == 3 else out[0]


@_on_tensor_device
def moe_quant_weight_int4(w: torch.Tensor):
    G, N, K = w.shape
    dev = w.device
    q = torch.empty((G, N, K // 2), dtype=torch.uint8, device=dev)
    s = torch.empty((G, N, K // 128), dtype=torch.float32, device=dev)
    _lib.check(_lib_().moe_quant_weight_int4(_ptr(w), G, N, K, _ptr(q), _ptr(s), _stream(dev)),
               "moe_quant_weight_int4")
    return q, s


@_on_tensor_device
def moe_pack_weight_int4(q: torch.Tensor, s7: torch.Tensor):
    """int4 codes [G, N, K/2] + scales [G, N, K/128] (moe_quant_weight_int4) -> the
    fragment-major order grouped_gemm_w4a8 reads (same shapes and byte counts)."""
    G, N, K2 = q.shape
    qf = torch.empty_like(q)
    s7f = torch.empty_like(s7)
    _lib.check(_lib_().moe_pack_weight_int4(_ptr(q), _ptr(s7), G, N, 2 * K2, _ptr(qf), _ptr(s7f),
                                            _stream(q.device)), "moe_pack_weight_int4")
    return qf, s7f


# --------------------------------------------------------------- grouped GEMM

@_on_tensor_device
def grouped_gemm_fp8(A, sA, B, sB, offsets, R_cap: int, N: int, swiglu: bool = False,
                     a_rows: Optional[torch.Tensor] = None, a_row_div: int = 1):
    """B: weight codes packed by moe_pack_weight_fp8.  Returns C bf16 [R_cap, N] (plain)
    or (codes e4m3 [R_cap, N], sC [R_cap, N/128])."""
    K = A.shape[1]
    G = B.shape[0]
    dev = A.device
    if swiglu:
        Cc = torch.empty((R_cap, N), dtype=torch.uint8, device=dev)
        sC = torch.empty((R_cap, N // 128), dtype=torch.float32, device=dev)
        out_dt, epi = MOE_E4M3, MOE_EPI_SWIGLU
    else:
        Cc = torch.empty((R_cap, N), dtype=torch.bfloat16, device=dev)
        sC = None
        out_dt, epi = MOE_BF16, MOE_EPI_PLAIN
    _lib.check(_lib_().grouped_gemm_fp8(_ptr(A), _ptr(sA), _ptr(a_rows), a_row_div, _ptr(B),
                                        _ptr(sB), _ptr(offsets), G, R_cap, N, K, epi, out_dt,
                                        _ptr(Cc), _ptr(sC), _stream(dev)), "grouped_gemm_fp8")
    return (Cc, sC) if swiglu else Cc


@_on_tensor_device
def grouped_gemm_w4a8(A, sA, B, s7, offsets, R_cap: int, N: int, swiglu: bool = False,
                      a_rows: Optional[torch.Tensor] = None, a_row_div: int = 1):
    """4-bit weights (packed by moe_pack_weight_int4) on the FP8 matrix core.  Returns C bf16
    [R_cap, N] (plain) or (codes e4m3 [R_cap, N], sC [R_cap, N/128])."""
    K = A.shape[1]
    G = B.shape[0]
    dev = A.device
    if swiglu:
        Cc = torch.empty((R_cap, N), dtype=torch.uint8, device=dev)
        sC = torch.empty((R_cap, N // 128), dtype=torch.float32, device=dev)
        out_dt, epi = MOE_E4M3, MOE_EPI_SWIGLU
    else:
        Cc = torch.empty((R_cap, N), dtype=torch.bfloat16, device=dev)
        sC = None
        out_dt, epi = MOE_BF16, MOE_EPI_PLAIN
    _lib.check(_lib_().grouped_gemm_w4a8(_ptr(A), _ptr(sA), _ptr(a_rows), a_row_div, _ptr(B),
                                         _ptr(s7), _ptr(offsets), G, R_cap, N, K, epi, out_dt,
                                         _ptr(Cc), _ptr(sC), _stream(dev)), "grouped_gemm_w4a8")
    return (Cc, sC) if swiglu else Cc


@_on_tensor_device
def grouped_gemm_fp8_masked(A, sA, B, sB, counts, cap: int, N: int, swiglu: bool = False):
    """Fixed-capacity layout: A [G*cap, K]; group g owns rows [g*cap, g*cap + counts[g]).
    Returns C bf16 [G*cap, N] (plain) or (codes e4m3 [G*cap, N], sC [G*cap, N/128])."""
    K = A.shape[1]
    G = B.shape[0]
    dev = A.device
    rows = G * cap
    if swiglu:
        Cc = torch.empty((rows, N), dtype=torch.uint8, device=dev)
        sC = torch.empty((rows, N // 128), dtype=torch.float32, device=dev)
        out_dt, epi = MOE_E4M3, MOE_EPI_SWIGLU
    else:
        Cc = torch.empty((rows, N), dtype=torch.bfloat16, device=dev)
        sC = None
        out_dt, epi = MOE_BF16, MOE_EPI_PLAIN
    _lib.check(_lib_().grouped_gemm_fp8_masked(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(counts),
                                               G, cap, N, K, epi, out_dt, _ptr(Cc), _ptr(sC),
                                               _stream(dev)), "grouped_gemm_fp8_masked")
    return (Cc, sC) if swiglu else Cc


@_on_tensor_device
def gemm_fp8(A, sA, B, sB):
    """Dense block-scaled FP8 GEMM: A [M, K] e4m3 + sA, B [N, K] e4m3 codes packed by
    moe_pack_weight_fp8 + sB -> bf16 [M, N]."""
    M, K = A.shape
    N = B.shape[0]
    Cc = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _lib.check(_lib_().gemm_fp8(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), M, N, K, _ptr(Cc),
                                _stream(A.device)), "gemm_fp8")
    return Cc


@_on_tensor_device
def grouped_gemm_w4a16(A, B, s7, offsets, R_cap: int, N: int, swiglu: bool = False,
                       a_rows: Optional[torch.Tensor] = None, a_row_div: int = 1):
    K = A.shape[1]
    G = B.shape[0]
    dev = A.device
    Cc = torch.empty((R_cap, N), dtype=torch.bfloat16, device=dev)
    _lib.check(_lib_().grouped_gemm_w4a16(_ptr(A), _ptr(a_rows), a_row_div, _ptr(B), _ptr(s7),
                                          _ptr(offsets), G, R_cap, N, K,
                                          MOE_EPI_SWIGLU if swiglu else MOE_EPI_PLAIN, _ptr(Cc),
                                          _stream(dev)), "grouped_gemm_w4a16")
    return Cc


@_on_tensor_device
def grouped_gemm_f32(A, B, offsets, R_cap: int, N: int, swiglu: bool = False,
                     a_rows: Optional[torch.Tensor] = None, a_row_div: int = 1):
    K = A.shape[1]
    G = B.shape[0]
    dev = A.device
    Cc = torch.empty((R_cap, N), dtype=torch.float32, device=dev)
    _lib.check(_lib_().grouped_gemm_f32(_ptr(A), _ptr(a_rows), a_row_div, _ptr(B), _ptr(offsets),
                                        G, R_cap, N, K,
                                        MOE_EPI_SWIGLU if swiglu else MOE_EPI_PLAIN, _ptr(Cc),
                                        _stream(dev)), "grouped_gemm_f32")
    return Cc


@_on_tensor_device
def moe_combine(o: torch.Tensor, row_of_slot: torch.Tensor, topk_w: torch.Tensor, T: int, k: int,
                out_dtype=torch.bfloat16):
    d = o.shape[1]
    dev = o.device
    y = torch.empty((T, d), dtype=out_dtype, device=dev)
    _lib.check(_lib_().moe_combine(_ptr(o), _dt(o), _ptr(row_of_slot), _ptr(topk_w), T, k, d,
                                   _ptr(y), _dt(y), _stream(dev)), "moe_combine")
    return y


# ------------------------------------------- few tokens with 4-bit expert weights

def _want(fn: str, name: str, t: Optional[torch.Tensor], dtype, *shape):
    """Refuse a tensor of another dtype or shape than the call takes (None passes)."""
    if t is not None and (t.dtype != dtype or t.shape != shape):
        raise ValueError(f"{fn}: {name} must be {dtype} {list(shape)}, got {t.dtype} "
                         f"{list(t.shape)}")


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _int4_weight(fn: str, name: str, q: torch.Tensor, s7: torch.Tensor):
    """(G, rows, K, group) of int4 codes [G, rows, K/2] and scales [G, rows, K/group]."""
    if q.dim() != 3 or s7.dim() != 3 or q.dtype != torch.uint8 or s7.dtype != torch.float32 \
            or q.shape[:2] != s7.shape[:2] or s7.shape[2] == 0 \
            or (2 * q.shape[2]) % s7.shape[2]:
        raise ValueError(f"{fn}: {name} must be uint8 codes [G, rows, K/2] with fp32 scales "
                         f"[G, rows, K/group], got {q.dtype} {list(q.shape)} and {s7.dtype} "
                         f"{list(s7.shape)}")
    K = 2 * q.shape[2]
    return q.shape[0], q.shape[1], K, K // s7.shape[2]


@_on_tensor_device
def moe_quant_weight_int4_group(w: torch.Tensor, group: int):
    """fp32 weights [G, N, K] -> int4 codes [G, N, K/2] and scales [G, N, K/group], one scale
    per `group` (32, 64 or 128) weights of a row."""
    fn = "moe_quant_weight_int4_group"
    G, N, K = w.shape
    if w.dtype != torch.float32 or group not in (32, 64, 128) or K % group:
        raise ValueError(f"{fn}: w must be fp32 with K a multiple of group (32, 64 or 128), got "
                         f"{w.dtype}, K = {K}, group = {group}")
    q = torch.empty((G, N, K // 2), dtype=torch.uint8, device=w.device)
    s7 = torch.empty((G, N, K // group), dtype=torch.float32, device=w.device)
    _lib.check(_lib_().moe_quant_weight_int4_group(_ptr(w), G, N, K, group, _ptr(q), _ptr(s7),
                                                   _stream(w.device)), fn)
    return q, s7


@_on_tensor_device
def moe_matvec_int4(x: torch.Tensor, q: torch.Tensor, s7: torch.Tensor,
                    idx: Optional[torch.Tensor] = None, x_div: int = 1, swiglu: bool = False,
                    out_dtype: Optional[torch.dtype] = None):
    """Products of a few rows x [rows, K] with int4 weights q [G, Nb, K/2], s7 [G, Nb,
    K/group].  Slot s takes row s // x_div and expert idx[s] (int32 [S]; rows of slots whose
    expert lies outside [0, G) are zeros); without idx every row takes matrix 0 (x_div 1).
    Returns y [S, N] of out_dtype (x's by default), N = Nb or, with swiglu, Nb / 2."""
    fn = "moe_matvec_int4"
    G, rows, K, group = _int4_weight(fn, "q, s7", q, s7)
    if swiglu and rows % 2:
        raise ValueError(f"{fn}: swiglu needs an even number of weight rows, got {rows}")
    N = rows // 2 if swiglu else rows
    if x_div < 1:
        raise ValueError(f"{fn}: x_div must be >= 1")
    if idx is None:
        if x_div != 1:
            raise ValueError(f"{fn}: x_div needs idx")
        S = x.shape[0]
    else:
        S = idx.numel()
        _want(fn, "idx", idx, torch.int32, S)
    _want(fn, "x", x, x.dtype, (S + x_div - 1) // x_div, K)
    x_dt = _dt(x)
    y = torch.empty((S, N), dtype=out_dtype or x.dtype, device=x.device)
    _lib.check(_lib_().moe_matvec_int4(_ptr(x), x_dt, x_div, _ptr(q), _ptr(s7), group,
                                       _ptr(idx), S, G, N, K,
                                       MOE_EPI_SWIGLU if swiglu else MOE_EPI_PLAIN, _ptr(y),
                                       _dt(y), _stream(x.device)), fn)
    return y


def moe_ffn_int4_workspace_size(T: int, k: int, d: int, I: int) -> int:
    return _lib_().moe_ffn_int4_workspace_size(T, k, d, I)


@_on_tensor_device
def moe_ffn_int4(x: torch.Tensor, w13: torch.Tensor, s13: torch.Tensor, w2: torch.Tensor,
                 s2: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                 workspace: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """The routed experts' FFN of a few tokens x [T, d] with int4 weights w13 [E, 2I, d/2]
    (gate rows, then up rows) and w2 [E, d, I/2], after moe_route: the weighted sum over each
    token's experts topk_idx [T, k].  Returns y [T, d] of x's dtype."""
    fn = "moe_ffn_int4"
    E, rows, d, group = _int4_weight(fn, "w13, s13", w13, s13)
    I = rows // 2
    T, k = topk_idx.shape
    if _int4_weight(fn, "w2, s2", w2, s2) != (E, d, I, group) or rows % 2:
        raise ValueError(f"{fn}: w13 {list(w13.shape)} and w2 {list(w2.shape)} must be "
                         "[E, 2I, d/2] and [E, d, I/2] with the same group")
    _want(fn, "x", x, x.dtype, T, d)
    _want(fn, "topk_idx", topk_idx, torch.int32, T, k)
    _want(fn, "topk_w", topk_w, torch.float32, T, k)
    dt = _dt(x)
    if y is None:
        y = torch.empty((T, d), dtype=x.dtype, device=x.device)
    _want(fn, "y", y, x.dtype, T, d)
    if workspace is None:
        workspace = torch.empty(moe_ffn_int4_workspace_size(T, k, d, I), dtype=torch.uint8,
                                device=x.device)
    _lib.check(_lib_().moe_ffn_int4(_ptr(x), dt, _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2),
                                    group, _ptr(topk_idx), _ptr(topk_w), T, k, E, d, I, _ptr(y),
                                    _ptr(workspace), _nbytes(workspace), _stream(x.device)), fn)
    return y


# --------------------------------------------------- the router's training side

def moe_balance_workspace_size(T: int, E: int, B: int = 1) -> int:
    return _lib_().moe_balance_workspace_size(T, E, B)


def moe_route_bwd_workspace_size(T: int, E: int) -> int:
    return _lib_().moe_route_bwd_workspace_size(T, E)


_BALANCE_KINDS = {"switch": _lib.MOE_BALANCE_SWITCH, "square": _lib.MOE_BALANCE_SQUARE}


def _router_args(fn, logits, topk_idx, bias, mask, offsets):
    T, E = logits.shape
    B = 1 if offsets is None else offsets.numel() - 1
    k = topk_idx.shape[1] if topk_idx is not None else 1
    _want(fn, "logits", logits, torch.float32, T, E)
    _want(fn, "topk_idx", topk_idx, torch.int32, T, k)
    _want(fn, "bias", bias, torch.float32, E)
    _want(fn, "offsets", offsets, torch.int32, B + 1)
    if mask is not None:                                # a bool is a byte
        _want(fn, "mask", mask, torch.bool if mask.dtype == torch.bool else torch.uint8, T)
    return T, E, k, B


@_on_tensor_device
def moe_balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor,
                     bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                     offsets: Optional[torch.Tensor] = None, coef: float = 0.01,
                     kind: str = "switch", workspace: Optional[torch.Tensor] = None):
    """Load-balance loss of a routed batch (logits [T, E], topk_idx [T, k] of moe_route), over
    the segments offsets [B+1] (int32; None: the whole batch) and the tokens whose mask byte
    is nonzero.  kind "switch": coef E sum f_e P_e; "square": coef sum (P_e - 1/E)^2.
    Returns (loss [], counts [B, E], probs [B, E], grad [B, E]); grad goes to moe_route_bwd."""
    fn = "moe_balance_loss"
    if kind not in _BALANCE_KINDS:
        raise ValueError(f"{fn}: kind must be one of {sorted(_BALANCE_KINDS)}, got {kind!r}")
    T, E, k, B = _router_args(fn, logits, topk_idx, bias, mask, offsets)
    dev = logits.device
    counts = torch.empty((B, E), dtype=torch.int32, device=dev)
    probs = torch.empty((B, E), dtype=torch.float32, device=dev)
    grad = torch.empty((B, E), dtype=torch.float32, device=dev)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(moe_balance_workspace_size(T, E, B), dtype=torch.uint8, device=dev)
    _lib.check(_lib_().moe_balance_loss(_ptr(logits), _ptr(bias), _ptr(topk_idx), _ptr(mask),
                                        _ptr(offsets), T, E, k, B, _BALANCE_KINDS[kind], coef,
                                        counts.data_ptr(), probs.data_ptr(), grad.data_ptr(),
                                        loss.data_ptr(), _ptr(workspace), _nbytes(workspace),
                                        _stream(dev)), fn)
    return loss, counts, probs, grad


@_on_tensor_device
def moe_route_bwd(logits: torch.Tensor, topk_idx: Optional[torch.Tensor] = None,
                  dtopk_w: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  renorm: bool = False, mask: Optional[torch.Tensor] = None,
                  offsets: Optional[torch.Tensor] = None,
                  balance_grad: Optional[torch.Tensor] = None,
                  dloss: Optional[torch.Tensor] = None, need_dbias: bool = False,
                  workspace: Optional[torch.Tensor] = None):
    """Gradient of moe_route's gate weights (dtopk_w [T, k]) and of moe_balance_loss
    (balance_grad [B, E], its upstream gradient dloss, one fp32 on the GPU, 1 if None) with
    respect to the logits.  Returns dlogits [T, E], or (dlogits, dbias [E]) with need_dbias."""
    fn = "moe_route_bwd"
    T, E, k, B = _router_args(fn, logits, topk_idx, bias, mask, offsets)
    dev = logits.device
    _want(fn, "dtopk_w", dtopk_w, torch.float32, T, k)
    _want(fn, "balance_grad", balance_grad, torch.float32, B, E)
    if dloss is not None and (dloss.dtype != torch.float32 or dloss.numel() != 1):
        raise ValueError(f"{fn}: dloss must be one fp32 value")
    dlogits = torch.empty((T, E), dtype=torch.float32, device=dev)
    dbias = torch.empty(E, dtype=torch.float32, device=dev) if need_dbias else None
    if need_dbias and workspace is None:
        workspace = torch.empty(moe_route_bwd_workspace_size(T, E), dtype=torch.uint8, device=dev)
    _lib.check(_lib_().moe_route_bwd(_ptr(logits), _ptr(bias), _ptr(topk_idx), _ptr(dtopk_w),
                                     _ptr(mask), _ptr(offsets), _ptr(balance_grad), _ptr(dloss),
                                     T, E, k, B, MOE_ROUTE_RENORM if renorm else 0, _ptr(dlogits),
                                     _ptr(dbias), _ptr(workspace),
                                     _nbytes(workspace),
                                     _stream(dev)), fn)
    return (dlogits, dbias) if need_dbias else dlogits


# --------------------------------------------------------- measurement probes

def moe_probe_mfma_fp8(n_blocks: int, iters: int, code: int = 0x38,
                       device: Optional[torch.device] = None):
    """Enqueue the FP8 matrix-core probe on the current stream of `device` (default
    cuda:0); returns its fp32 output [n_blocks * 512] (n_blocks * 8 * iters * 4 * 65536
    FLOP are performed)."""
    dev = torch.device(device or "cuda:0")
    out = torch.empty(n_blocks * 512, dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _lib.check(_lib_().moe_probe_mfma_fp8(n_blocks, iters, code, _ptr(out), _stream(dev)),
                   "moe_probe_mfma_fp8")
    return out


@_on_tensor_device
def moe_probe_hbm_read(buf: torch.Tensor, n_blocks: int):
    """Enqueue the HBM read probe over the bytes of `buf`; returns the per-workgroup
    XORs of the 32-bit words read (uint32 stored as int32) [n_blocks]."""
    dev = buf.device
    out = torch.empty(n_blocks, dtype=torch.int32, device=dev)
    nbytes = buf.numel() * buf.element_size()
    _lib.check(_lib_().moe_probe_hbm_read(_ptr(buf), nbytes, n_blocks, _ptr(out), _stream(dev)),
               "moe_probe_hbm_read")
    return out


# ---------------------------------------------------------------------- layer

class LayerDesc:
    """Python view of moe_layer_desc."""

    def __init__(self, T, d, E, k, I, mode="fp8", route="score", renorm=False,
                 capacity_factor=0.0, m_align=128, layout="contiguous"):
        modes = {"fp32": MOE_MODE_FP32, "fp8": MOE_MODE_FP8, "w4a16": MOE_MODE_W4A16,
                 "w4a8": MOE_MODE_W4A8}
        layouts = {"contiguous": _lib.MOE_LAYOUT_CONTIGUOUS, "masked": _lib.MOE_LAYOUT_MASKED}
        self.c = MoeLayerDesc(T, d, E, k, I, modes[mode],
                              MOE_ROUTE_HASH if route == "hash" else MOE_ROUTE_SCORE,
                              MOE_ROUTE_RENORM if renorm else 0, float(capacity_factor), m_align,
                              layouts[layout])


def moe_layer_workspace_size(desc: LayerDesc) -> int:
    n = _lib_().moe_layer_workspace_size(C.byref(desc.c))
    if n == 0:
        raise MoeError(_lib.MOE_ERR_INVALID_ARG, "moe_layer_workspace_size",
                       _lib_().moe_last_error().decode())
    return n


@_on_tensor_device
def moe_layer_fwd(desc: LayerDesc, weights: dict, x: torch.Tensor,
                  token_ids: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  y: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None):
    """Whole layer forward.  ``weights`` holds w_router, bias, w13, s13, w2, s2 tensors
    (as moe_layer_weights).  Returns (y, counts)."""
    dev = x.device
    ws_bytes = moe_layer_workspace_size(desc)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    if counts is None:
        counts = torch.empty(desc.c.E, dtype=torch.int32, device=dev)
    w = MoeLayerWeights(*(_ptr(weights.get(n)) for n in ("w_router", "bias", "w13", "s13", "w2",
                                                        "s2")))
    _lib.check(_lib_().moe_layer_fwd(C.byref(desc.c), C.byref(w), _ptr(x), _ptr(token_ids),
                                     _ptr(y), _ptr(workspace), workspace.numel(), _ptr(counts),
                                     _stream(dev)), "moe_layer_fwd")
    return y, counts


def moe_layer_chunked_workspace_size(desc: LayerDesc, chunk_tokens: int) -> int:
    n = _lib_().moe_layer_chunked_workspace_size(C.byref(desc.c), chunk_tokens)
    if n == 0:
        raise MoeError(_lib.MOE_ERR_INVALID_ARG, "moe_layer_chunked_workspace_size",
                       _lib_().moe_last_error().decode() or "chunked pipeline not available "
                       "for this descriptor")
    return n


@_on_tensor_device
def moe_layer_fwd_chunked(desc: LayerDesc, weights: dict, x: torch.Tensor, chunk_tokens: int,
                          token_ids: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None,
                          y: Optional[torch.Tensor] = None,
                          aux_stream: Optional[torch.cuda.Stream] = None):
    """The layer forward as a two-stream chunk pipeline (chunk i's routing, dispatch and
    quantisation on ``aux_stream`` beside chunk i-1's GEMMs on the current stream).
    Returns y."""
    dev = x.device
    if workspace is None:
        workspace = torch.empty(moe_layer_chunked_workspace_size(desc, chunk_tokens),
                                dtype=torch.uint8, device=dev)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    if aux_stream is None:
        aux_stream = torch.cuda.Stream(device=dev)
    w = MoeLayerWeights(*(_ptr(weights.get(n)) for n in ("w_router", "bias", "w13", "s13", "w2",
                                                        "s2")))
    _lib.check(_lib_().moe_layer_fwd_chunked(C.byref(desc.c), C.byref(w), _ptr(x),
                                             _ptr(token_ids), _ptr(y), _ptr(workspace),
                                             workspace.numel(), chunk_tokens, _stream(dev),
                                             C.c_void_p(aux_stream.cuda_stream)),
               "moe_layer_fwd_chunked")
    return y
