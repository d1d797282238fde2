"""Cases of the router's balance loss and backward pass and of the few-token products with
4-bit expert weights: their inputs, plain forms and 64-bit values.

A case's ``op`` names the operator: ``matvec`` (moe_matvec_int4), ``ffn`` (moe_ffn_int4),
``balance`` (moe_balance_loss) or ``bwd`` (moe_route_bwd).  ``run`` computes it with
elementary torch operations, or, where ``own`` is true, with the library's kernels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------ cases

def _matvec(name, T, k, G, N, K, group, x, y, swiglu, dropped=0):
    return {"name": name, "op": "matvec", "T": T, "k": k, "G": G, "N": N, "K": K,
            "group": group, "x": x, "y": y, "swiglu": swiglu, "dropped": dropped}


def _ffn(name, T, k, E, d, I, group, x, dropped=0):
    return {"name": name, "op": "ffn", "T": T, "k": k, "E": E, "d": d, "I": I,
            "group": group, "x": x, "dropped": dropped}


def _balance(name, T, E, k, B, masked, kind, bias):
    return {"name": name, "op": "balance", "T": T, "E": E, "k": k, "B": B,
            "masked": masked, "kind": kind, "bias": bias}


def _bwd(name, T, E, k, B, masked, renorm, gate, balance, dbias):
    return {"name": name, "op": "bwd", "T": T, "E": E, "k": k, "B": B, "masked": masked,
            "renorm": renorm, "gate": gate, "balance": balance, "dbias": dbias}


def listed():
    return [
        # one token through one projection whose weights every token uses (a shared
        # expert's down projection at the decode layer's sizes)
        _matvec("matvec_one_token", 1, 0, 1, 7168, 2048, 128, "bf16", "bf16", False),
        # a handful of tokens through an oddly sized projection, fp32, fine groups
        _matvec("matvec_odd_f32", 13, 0, 1, 1003, 4128, 32, "f32", "f32", False),
        # four sequences decoding: gate and up products of their 8 of 256 experts
        _matvec("matvec_routed_swiglu", 4, 8, 256, 2048, 7168, 128, "bf16", "f32", True),
        # one sequence decoding: the experts' whole FFN of one token
        _ffn("ffn_one_token", 1, 8, 256, 7168, 2048, 128, "bf16"),
        # a small decode batch, one of its rows padding
        _ffn("ffn_batch_16", 16, 8, 256, 7168, 2048, 128, "bf16", 8),
        # hash-routed layer (one expert a token), 64-wide groups
        _ffn("ffn_hash_24", 24, 1, 64, 4096, 2048, 64, "bf16"),
        # the tiny fp32 layer: launch latency
        _ffn("ffn_tiny_f32", 3, 2, 8, 256, 512, 32, "f32", 1),
        # load statistics of one decode step
        _balance("balance_decode", 128, 256, 8, 1, False, "switch", True),
        # ragged sequences of a prefill batch, padding tokens masked
        _balance("balance_prefill", 4096, 256, 8, 9, True, "switch", True),
        # a training batch
        _balance("balance_train", 65536, 256, 8, 16, True, "square", False),
        # the router's backward pass at the prefill batch: gate weights, loss and bias
        _bwd("bwd_prefill", 4096, 256, 8, 9, True, False, True, True, True),
        # a training batch over 64 experts with renormalised gates
        _bwd("bwd_train", 131072, 64, 6, 16, False, True, True, True, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matvec", "ffn", "balance", "bwd"])
    group = rng.choice([32, 64, 128])
    x = rng.choice(["bf16", "bf16", "f32"])
    if op == "matvec":
        K = group * max(1, _log(rng, 128, 8192) // group)
        routed = rng.random() < 0.5
        G = rng.choice([8, 16, 64, 160]) if routed else 1
        T = _log(rng, 1, 16)
        k = rng.randint(1, 8) if routed else 0
        N = _log(rng, 17, 4096 if routed else 16384)
        return {"op": op, "T": T, "k": k, "G": G, "N": N, "K": K, "group": group, "x": x,
                "y": rng.choice(["bf16", "f32"]), "swiglu": rng.random() < 0.4,
                "dropped": rng.choice([0, 0, T * k // 3])}
    if op == "ffn":
        E = rng.choice([4, 8, 32, 64, 128])
        T = _log(rng, 1, 32)
        k = rng.randint(1, min(E, 8, max(1, 96 // T)))
        return {"op": op, "T": T, "k": k, "E": E, "d": 128 * rng.randint(1, 56),
                "I": 128 * rng.randint(1, 16), "group": group, "x": x,
                "dropped": rng.choice([0, 0, T * k // 4])}
    T = _log(rng, 1, 65536)
    E = rng.choice([4, 7, 33, 64, 100, 160, 256])
    k = rng.randint(1, min(E, 8))
    B = 1 if T < 64 or rng.random() < 0.4 else rng.randint(2, 24)
    masked = T >= 64 and rng.random() < 0.5
    if op == "balance":
        return {"op": op, "T": T, "E": E, "k": k, "B": B, "masked": masked,
                "kind": rng.choice(["switch", "square"]), "bias": rng.random() < 0.5}
    gate = rng.random() < 0.8
    return {"op": op, "T": T, "E": E, "k": k, "B": B, "masked": masked,
            "renorm": rng.random() < 0.5, "gate": gate,
            "balance": not gate or rng.random() < 0.6, "dbias": rng.random() < 0.5}


# ----------------------------------------------------------------------------- inputs

def _int4(g, G, N, K, group):
    """Codes evenly over the whole range and scales that give weights of about 1/sqrt(K)."""
    q = torch.randint(0, 256, (G, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.rand((G, N, K // group), generator=g, device="cuda")
    return q, s.add_(0.5).mul_(1.0 / (4.5 * math.sqrt(K)))


def _experts(g, T, k, E, dropped):
    """k different experts a token, int32 [T, k]; the last `dropped` slots hold -1."""
    idx = torch.rand((T, E), generator=g, device="cuda").argsort(dim=1)[:, :k]
    idx = idx.to(torch.int32).contiguous()
    if dropped:
        idx.view(-1)[-dropped:] = -1
    return idx


def _router(g, case):
    """Logits with a preference per expert, the experts that they choose, a mask and the
    first token of each ragged sequence (the last one ends before the batch does)."""
    T, E, k, B = case["T"], case["E"], case["k"], case["B"]
    z = torch.randn((T, E), generator=g, device="cuda")
    z += 0.5 * torch.randn((1, E), generator=g, device="cuda")
    b = 0.02 * torch.rand((E,), generator=g, device="cuda") - 0.01
    key = z + b if case.get("bias", True) else z
    idx = torch.topk(key, k, dim=1).indices.to(torch.int32).contiguous()
    state = {"logits": z, "bias": b if case.get("bias", True) else None, "idx": idx,
             "mask": None, "offsets": None, "B": B}
    if case["masked"]:
        state["mask"] = (torch.rand((T,), generator=g, device="cuda") < 0.9).to(torch.uint8)
    if B > 1:
        cut = torch.randint(0, T + 1, (B + 1,), generator=g, device="cuda").sort().values
        cut[0] = 0
        state["offsets"] = cut.to(torch.int32)
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    if op == "matvec":
        T, k, N, K = case["T"], case["k"], case["N"], case["K"]
        q, s = _int4(g, case["G"], 2 * N if case["swiglu"] else N, K, case["group"])
        x = torch.randn((T, K), generator=g, device="cuda").to(DTYPES[case["x"]])
        idx = _experts(g, T, k, case["G"], case["dropped"]).view(-1) if k else None
        return {"op": op, "x": x, "q": q, "s": s, "idx": idx, "div": max(k, 1),
                "swiglu": case["swiglu"], "y": DTYPES[case["y"]]}
    if op == "ffn":
        T, k, E, d, I = case["T"], case["k"], case["E"], case["d"], case["I"]
        w13, s13 = _int4(g, E, 2 * I, d, case["group"])
        w2, s2 = _int4(g, E, d, I, case["group"])
        x = torch.randn((T, d), generator=g, device="cuda").to(DTYPES[case["x"]])
        gate = torch.rand((T, k), generator=g, device="cuda")
        return {"op": op, "x": x, "w13": w13, "s13": s13, "w2": w2, "s2": s2,
                "idx": _experts(g, T, k, E, case["dropped"]), "w": gate / gate.sum(1, True)}
    state = _router(g, case)
    state["op"] = op
    if op == "balance":
        return state | {"kind": case["kind"], "coef": 0.01}
    T, E, k, B = case["T"], case["E"], case["k"], case["B"]
    dw = torch.randn((T, k), generator=g, device="cuda") if case["gate"] else None
    grad = dloss = None
    if case["balance"]:
        grad = torch.randn((B, E), generator=g, device="cuda")
        dloss = 0.5 + torch.rand((), generator=g, device="cuda")
    return state | {"dw": dw, "grad": grad, "dloss": dloss, "renorm": case["renorm"],
                    "dbias": case["dbias"]}


# ------------------------------------------------------------------------ plain forms

def _weights(q, s):
    """Packed codes [.., N, K/2] and scales [.., N, K/group] -> fp32 weights [.., N, K].
    Four bytes hold eight consecutive codes, byte b the codes b (low nibble) and 4 + b;
    a nibble is a sign (bit 3) and a magnitude."""
    low = (q & 7).float() * (1 - 2 * ((q >> 3) & 1).float())
    high = ((q >> 4) & 7).float() * (1 - 2 * (q >> 7).float())
    b4 = (*q.shape[:-1], q.shape[-1] // 4, 4)
    v = torch.stack((low.view(b4), high.view(b4)), dim=-2)
    v = v.view(*s.shape, -1) * s.unsqueeze(-1)
    return v.view(*q.shape[:-1], -1)


def _product(x, q, s, idx, swiglu):
    """Rows x [S, K] fp32 times each slot's expert; a slot without one gives zeros."""
    if idx is None:
        y = x @ _weights(q[0], s[0]).t()
    else:
        ok = (idx >= 0) & (idx < q.shape[0])
        e = torch.where(ok, idx, 0)
        y = torch.bmm(_weights(q[e], s[e]), x.unsqueeze(-1)).squeeze(-1)
        y = torch.where(ok[:, None], y, 0.0)
    if swiglu:
        gate, up = y.chunk(2, dim=1)
        y = gate / (1 + torch.exp(-gate)) * up
    return y


def _segments(st):
    """Sequence of each token, whether it counts, and how many of a sequence count."""
    T, dev = st["logits"].shape[0], st["logits"].device
    t = torch.arange(T, device=dev)
    ok = torch.ones(T, dtype=torch.bool, device=dev) if st["mask"] is None else st["mask"] != 0
    if st["offsets"] is None:
        seg = torch.zeros_like(t)
    else:
        off = st["offsets"].long()
        seg = torch.searchsorted(off[1:].contiguous(), t, right=True)
        ok = ok & (t >= off[0]) & (t < off[-1])
        seg = seg.clamp(max=st["B"] - 1)
    n = torch.zeros(st["B"], dtype=torch.float64, device=dev).index_add_(0, seg, ok.double())
    return seg, ok, n


def _softmax(st, ok):
    key = st["logits"] if st["bias"] is None else st["logits"] + st["bias"]
    e = torch.exp(key - key.max(dim=1, keepdim=True).values)
    return torch.where(ok[:, None], e / e.sum(dim=1, keepdim=True), 0.0)


def _plain_balance(st):
    B, k = st["B"], st["idx"].shape[1]
    E = st["logits"].shape[1]
    seg, ok, n = _segments(st)
    p = _softmax(st, ok)
    dev = p.device
    of = (torch.arange(B, device=dev)[:, None] == seg[None, :]).double()
    P = (of @ p.double()) / n.clamp(min=1)[:, None]
    slot = seg[:, None] * E + st["idx"]
    slot = torch.where(ok[:, None] & (st["idx"] >= 0), slot, B * E).view(-1)
    counts = torch.zeros(B * E + 1, dtype=torch.int64, device=dev)
    counts = counts.index_add_(0, slot, torch.ones_like(slot))[:-1].view(B, E)
    live = (n > 0).double()
    each = (live / (n.clamp(min=1) * live.sum().clamp(min=1)))[:, None]
    if st["kind"] == "switch":
        f = counts.double() / (k * n.clamp(min=1))[:, None]
        loss = E * (f * P).sum(dim=1)
        grad = E * (f - f.mean(dim=1, keepdim=True)) * each
    else:
        off = (P - 1.0 / E) * live[:, None]
        loss = off.square().sum(dim=1)
        grad = 2 * off * each
    loss = (loss * live).sum() / live.sum().clamp(min=1)
    c = st["coef"]
    return {"loss": (c * loss).float(), "counts": counts.int(), "probs": P.float(),
            "grad": (c * grad).float()}


def _plain_bwd(st):
    seg, ok, _ = _segments(st)
    p = _softmax(st, ok)
    G = torch.zeros_like(p)
    if st["grad"] is not None:
        G = st["dloss"] * st["grad"][seg]
    chosen = 0.0
    if st["dw"] is not None:
        at = st["idx"].long()
        dw = torch.where(ok[:, None], st["dw"], 0.0)
        if st["renorm"]:
            w = p.gather(1, at)
            w = torch.where(ok[:, None], w / w.sum(dim=1, keepdim=True), 0.0)
            a = w * (dw - (w * dw).sum(dim=1, keepdim=True))
            chosen = torch.zeros_like(p).scatter_add_(1, at, a)
        else:
            G = G.scatter_add(1, at, dw)
    dz = p * (G - (p * G).sum(dim=1, keepdim=True)) + chosen
    out = {"dlogits": dz}
    if st["dbias"]:
        out["dbias"] = dz.double().sum(dim=0).float()
    return out


def _plain(st):
    if st["op"] == "matvec":
        x = st["x"].float()
        if st["idx"] is not None:
            x = x.repeat_interleave(st["div"], dim=0)
        return _product(x, st["q"], st["s"], st["idx"], st["swiglu"]).to(st["y"])
    if st["op"] == "ffn":
        T, k = st["idx"].shape
        x = st["x"].float().repeat_interleave(k, dim=0)
        idx = st["idx"].view(-1)
        h = _product(x, st["w13"], st["s13"], idx, True)
        o = _product(h, st["w2"], st["s2"], idx, False)
        return (o.view(T, k, -1) * st["w"][:, :, None]).sum(dim=1).to(st["x"].dtype)
    return _plain_balance(st) if st["op"] == "balance" else _plain_bwd(st)


# ------------------------------------------------------------------------------- run

def run(state):
    if not own:
        return _plain(state)
    import fp8_grouped_gemm_amd as M
    st = state
    if st["op"] == "matvec":
        return M.moe_matvec_int4(st["x"], st["q"], st["s"], idx=st["idx"], x_div=st["div"],
                                 swiglu=st["swiglu"], out_dtype=st["y"])
    if st["op"] == "ffn":
        return M.moe_ffn_int4(st["x"], st["w13"], st["s13"], st["w2"], st["s2"], st["idx"],
                              st["w"])
    if st["op"] == "balance":
        loss, counts, probs, grad = M.moe_balance_loss(
            st["logits"], st["idx"], bias=st["bias"], mask=st["mask"], offsets=st["offsets"],
            coef=st["coef"], kind=st["kind"])
        return {"loss": loss, "counts": counts, "probs": probs, "grad": grad}
    got = M.moe_route_bwd(st["logits"], st["idx"], dtopk_w=st["dw"], bias=st["bias"],
                          renorm=st["renorm"], mask=st["mask"], offsets=st["offsets"],
                          balance_grad=st["grad"], dloss=st["dloss"], need_dbias=st["dbias"])
    return {"dlogits": got[0], "dbias": got[1]} if st["dbias"] else {"dlogits": got}


# ----------------------------------------------------------------------------- exact

def _exact_rows(x, q, s, group):
    """x [K] fp64 times one matrix, from the codes' meaning: a table of the 16 nibbles."""
    table = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, 0, -1, -2, -3, -4, -5, -6, -7],
                         dtype=torch.float64, device=q.device)
    N, K = q.shape[0], 2 * q.shape[1]
    byte = q.view(N, K // 8, 1, 4).long()
    v = table[torch.cat((byte & 15, byte >> 4), dim=2)].view(N, K) * x
    return (v.view(N, K // group, group).sum(dim=2) * s.double()).sum(dim=1)


def _silu(z):
    return z * 0.5 * (1.0 + torch.tanh(0.5 * z))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "matvec":
        x, N = st["x"].double(), case["N"]
        which = [0] * x.shape[0] if st["idx"] is None else st["idx"].tolist()
        rows = []
        for i, e in enumerate(which):
            if e < 0:
                rows.append(torch.zeros(N, dtype=torch.float64, device=x.device))
                continue
            r = _exact_rows(x[i // st["div"]], st["q"][e], st["s"][e], case["group"])
            rows.append(_silu(r[:N]) * r[N:] if case["swiglu"] else r)
        return torch.stack(rows)
    if op == "ffn":
        T, k, I = case["T"], case["k"], case["I"]
        y = torch.zeros((T, case["d"]), dtype=torch.float64, device="cuda")
        which = st["idx"].tolist()
        for t in range(T):
            for j in range(k):
                e = which[t][j]
                if e < 0:
                    continue
                r = _exact_rows(st["x"][t].double(), st["w13"][e], st["s13"][e], case["group"])
                h = _silu(r[:I]) * r[I:]
                o = _exact_rows(h, st["w2"][e], st["s2"][e], case["group"])
                y[t] += st["w"][t, j].double() * o
        return y

    # router: each sequence by itself, from the list of its tokens
    T, E, k, B = case["T"], case["E"], case["k"], case["B"]
    key = st["logits"] if st["bias"] is None else st["logits"] + st["bias"][None, :]
    logp = key.double() - torch.logsumexp(key.double(), dim=1, keepdim=True)
    cut = [0, T] if st["offsets"] is None else st["offsets"].tolist()
    keep = torch.ones(T, dtype=torch.bool) if st["mask"] is None else st["mask"].cpu() != 0
    lists = [torch.nonzero(keep[cut[b]:cut[b + 1]]).view(-1).cuda() + cut[b] for b in range(B)]
    live = sum(1 for v in lists if len(v))
    f64 = {"dtype": torch.float64, "device": "cuda"}
    if op == "balance":
        loss = 0.0
        counts = torch.zeros((B, E), dtype=torch.int64, device="cuda")
        probs, grad = torch.zeros((B, E), **f64), torch.zeros((B, E), **f64)
        for b, v in enumerate(lists):
            n = len(v)
            if n == 0:
                continue
            counts[b] = torch.bincount(st["idx"][v].view(-1).long(), minlength=E)
            probs[b] = torch.exp(logp[v]).mean(dim=0)
            if case["kind"] == "switch":
                f = counts[b].double() / (n * k)
                loss = loss + E * torch.dot(f, probs[b])
                grad[b] = E * (f - 1.0 / E) / (n * live)
            else:
                d = probs[b] - 1.0 / E
                loss = loss + torch.dot(d, d)
                grad[b] = 2 * d / (n * live)
        c = st["coef"]
        loss = c * torch.as_tensor(loss, **f64) / max(live, 1)
        return {"loss": loss, "counts": None, "probs": probs, "grad": c * grad}
    dz = torch.zeros((T, E), **f64)
    for b, v in enumerate(lists):
        p, i = torch.exp(logp[v]), st["idx"][v].long()
        if st["grad"] is not None:
            g = st["dloss"].double() * st["grad"][b].double()
            dz[v] += p * (g[None, :] - (p @ g)[:, None])
        if st["dw"] is None:
            continue
        dw = st["dw"][v].double()
        w = torch.gather(p, 1, i)
        if st["renorm"]:
            w = w / w.sum(dim=1, keepdim=True)
            mean = (w * dw).sum(dim=1, keepdim=True)
            dz[v] = dz[v].scatter_add(1, i, w * (dw - mean))
        else:
            mean = (w * dw).sum(dim=1, keepdim=True)
            dz[v] = dz[v].scatter_add(1, i, w * dw) - p * mean
    return {"dlogits": dz, "dbias": dz.sum(dim=0)} if case["dbias"] else {"dlogits": dz}


# ------------------------------------------------------------------------------ work

def _distinct(slots, G):
    """Experts that this many evenly spread slots touch, on average."""
    return G * (1.0 - (1.0 - 1.0 / G) ** slots)


def _int4_bytes(N, K, group):
    return N * (K / 2 + 4.0 * K / group)


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "matvec":
        S = case["T"] * max(case["k"], 1) - case["dropped"]
        rows = case["N"] * (2 if case["swiglu"] else 1)
        mats = _distinct(S, case["G"]) if case["k"] else 1
        io = case["T"] * case["K"] * size[case["x"]] + S * case["N"] * size[case["y"]]
        return {"bytes": mats * _int4_bytes(rows, case["K"], case["group"]) + io,
                "flops": 2.0 * S * rows * case["K"]}
    if op == "ffn":
        T, d, I, group = case["T"], case["d"], case["I"], case["group"]
        S = T * case["k"] - case["dropped"]
        one = _int4_bytes(2 * I, d, group) + _int4_bytes(d, I, group)
        return {"bytes": _distinct(S, case["E"]) * one + 2 * T * d * size[case["x"]],
                "flops": 6.0 * S * d * I}
    T, E, k, B = case["T"], case["E"], case["k"], case["B"]
    read = 4.0 * T * E + 4.0 * T * k + (T if case["masked"] else 0)
    if op == "balance":
        return {"bytes": read + 12.0 * B * E, "flops": 6.0 * T * E}
    wrote = 4.0 * T * E + (4.0 * E if case["dbias"] else 0)
    gate = 4.0 * T * k if case["gate"] else 0.0
    return {"bytes": read + wrote + gate + (4.0 * B * E if case["balance"] else 0),
            "flops": 10.0 * T * E}
