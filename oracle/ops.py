"""The operators beside the layer forward, in fp64 numpy (oracle side): products of a few
rows with 4-bit weights and group scales, the experts' FFN on them, the load-balance loss
and the router's backward pass.

The weights are the block-wise 4-bit codes of the DeepSeek-V4 lecture (tqpw.cn, sec. 3.1);
the FFN is y = sum_i G(x)_i E_i(x) with SwiGLU experts (discosf.com, sec. 2.1-2.2); the
router is the biased softmax of discosf.com sec. 2.2; the square loss is the
sum (p_i - 1/N)^2 form of the auxiliary losses the pages list, the other the product of an
expert's share of the slots and its mean probability (parity unpinned: the pages print no
values for either).
"""
from __future__ import annotations

import numpy as np


def int4_unpack(packed) -> np.ndarray:
    """Bytes [..., K/2] -> codes int8 [..., K] (the inverse of codecs.int4_pack; nibble 8,
    a negative zero, is 0)."""
    p = np.asarray(packed, np.uint8)
    w = p.reshape(*p.shape[:-1], -1, 4)
    nib = np.stack([w & 15, w >> 4], axis=-2).reshape(*p.shape[:-1], -1)
    mag = (nib & 7).astype(np.int8)
    return np.where(nib & 8, -mag, mag).astype(np.int8)


def int4_quant_group(w, group: int):
    """codecs.int4_quant_rows with blocks of `group` weights: codes int8 and scales."""
    w = np.asarray(w, np.float32)
    G, N, K = w.shape
    wb = w.reshape(G, N, K // group, group)
    amax = np.max(np.abs(wb), axis=3)
    amax = np.where(amax == 0, np.float32(1.0), amax).astype(np.float32)
    t = ((wb / amax[..., None]).astype(np.float32) * np.float32(7.0)).astype(np.float32)
    return (np.rint(t.astype(np.float64)).astype(np.int8).reshape(G, N, K),
            (amax / np.float32(7.0)).astype(np.float32))


def int4_weight(packed, s7) -> np.ndarray:
    """codes times scales, fp64 [G, N, K]."""
    q = int4_unpack(packed).astype(np.float64)
    group = q.shape[-1] // s7.shape[-1]
    return q * np.repeat(np.asarray(s7, np.float64), group, axis=-1)


def silu(z):
    return z * 0.5 * (1.0 + np.tanh(0.5 * z))


def matvec_int4(x, w, idx, x_div: int):
    """v [S, rows] of weights w [G, rows, K] and the sums of absolute terms beside it; a slot
    whose expert lies outside [0, G) gives zeros."""
    x = np.asarray(x, np.float64)
    G = w.shape[0]
    idx = [0] * x.shape[0] if idx is None else [int(i) for i in idx]
    v = np.zeros((len(idx), w.shape[1]))
    a = np.zeros_like(v)
    for s, e in enumerate(idx):
        if 0 <= e < G:
            v[s] = w[e] @ x[s // x_div]
            a[s] = np.abs(w[e]) @ np.abs(x[s // x_div])
    return v, a


def _counting(T, mask, offsets):
    """Token lists of the segments: inside, and mask nonzero."""
    keep = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    off = [0, T] if offsets is None else [int(o) for o in offsets]
    return [np.arange(off[b], off[b + 1])[keep[off[b]:off[b + 1]]] for b in range(len(off) - 1)]


def softmax_rows(logits, bias):
    """fp64 softmax of the fp32 keys; a row of -inf gives zeros."""
    key = np.asarray(logits, np.float32)
    if bias is not None:
        key = (key + np.asarray(bias, np.float32)[None, :]).astype(np.float32)
    key = key.astype(np.float64)
    with np.errstate(invalid="ignore"):
        m = key.max(axis=1, keepdims=True) if key.size else np.zeros((len(key), 1))
        z = np.exp(key - np.where(np.isneginf(m), 0.0, m))
        s = z.sum(axis=1, keepdims=True)
        return np.where(s == 0, 0.0, z / np.where(s == 0, 1.0, s))


def balance_loss(logits, topk_idx, bias=None, mask=None, offsets=None, coef=0.01, kind="switch"):
    """(loss, counts [B, E], probs [B, E], grad [B, E]); grad is dloss/dp of one counting
    token of the segment, less its mean over the experts for "switch"."""
    logits = np.asarray(logits, np.float32)
    T, E = logits.shape
    idx = np.asarray(topk_idx).reshape(T, -1)
    k = idx.shape[1]
    segs = _counting(T, mask, offsets)
    B = len(segs)
    counts = np.zeros((B, E), np.int64)
    probs, grad, loss = np.zeros((B, E)), np.zeros((B, E)), 0.0
    live = sum(len(s) > 0 for s in segs)
    for b, s in enumerate(segs):
        if not len(s):
            continue
        n = len(s)
        i = idx[s].ravel()
        counts[b] = np.bincount(i[(i >= 0) & (i < E)], minlength=E)
        probs[b] = softmax_rows(logits[s], bias).mean(axis=0)
        f = counts[b] / (k * n)
        if kind == "switch":
            loss += coef * E * np.sum(f * probs[b]) / live
            grad[b] = coef * E * (f - f.mean()) / (n * live)
        else:
            loss += coef * np.sum((probs[b] - 1 / E) ** 2) / live
            grad[b] = 2 * coef * (probs[b] - 1 / E) / (n * live)
    return loss, counts, probs, grad


def gate_weights(logits, topk_idx, bias=None, renorm=False):
    """The gate weights of given experts (fp64); slots without one have weight 0."""
    p = softmax_rows(logits, bias)
    idx = np.asarray(topk_idx)
    ok = (idx >= 0) & (idx < p.shape[1])
    w = np.where(ok, np.take_along_axis(p, np.where(ok, idx, 0), axis=1), 0.0)
    if renorm:
        s = w.sum(axis=1, keepdims=True)
        w = np.where(s == 0, 0.0, w / np.where(s == 0, 1.0, s))
    return w, p, ok


def route_bwd(logits, topk_idx, dtopk_w=None, bias=None, renorm=False, mask=None, offsets=None,
              balance_grad=None, dloss=1.0):
    """dlogits [T, E] and, beside it, the sums of the absolute values of its terms."""
    logits = np.asarray(logits, np.float32)
    T, E = logits.shape
    dz, mag = np.zeros((T, E)), np.zeros((T, E))
    for b, s in enumerate(_counting(T, mask, offsets)):
        if not len(s):
            continue
        p = softmax_rows(logits[s], bias)
        if balance_grad is not None:
            g = float(dloss) * np.asarray(balance_grad[b], np.float64)[None, :]
            dz[s] += p * (g - (p * g).sum(axis=1, keepdims=True))
            mag[s] += p * (np.abs(g) + (p * np.abs(g)).sum(axis=1, keepdims=True))
        if dtopk_w is None:
            continue
        idx = np.asarray(topk_idx)[s]
        w, _, ok = gate_weights(logits[s], idx, bias, renorm)
        dw = np.where(ok, np.asarray(dtopk_w, np.float64)[s], 0.0)
        mean = (w * dw).sum(axis=1, keepdims=True)
        amean = (w * np.abs(dw)).sum(axis=1, keepdims=True)
        rows = np.arange(len(s))[:, None] + 0 * idx
        at = np.where(ok, idx, 0)
        if renorm:
            np.add.at(dz, (s[rows], at), np.where(ok, w * (dw - mean), 0.0))
            np.add.at(mag, (s[rows], at), np.where(ok, w * (np.abs(dw) + amean), 0.0))
        else:
            np.add.at(dz, (s[rows], at), w * dw)
            np.add.at(mag, (s[rows], at), w * np.abs(dw))
            dz[s] -= p * mean
            mag[s] += p * amean
    return dz, mag
