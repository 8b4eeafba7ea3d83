"""Window attention with sinks, and chunk attention over a paged cache: cases to measure.

Four operators of the framework, each with its plain form in elementary torch operations:

forward  causal attention of every token t over the last `window` tokens and the first `sinks` tokens
         (A_t = {u <= t : t - u < window or u < sinks}); outputs h and lse.
train    the same forward and its backward for an upstream gradient g; outputs h, lse, dQ, dK, dV.
append   the new keys and values of a ragged batch written into their pages; outputs both caches.
attend   the new tokens of a ragged batch over a paged cache (window and sinks as above); outputs h and lse.
"""
import math

import torch

own = False

EVERYTHING = 2**31 - 1  # a window that hides nothing
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # prompt pass of a small model: head dim 64, 16 query heads to a kv head, a 256-token window
        dict(name="forward small model", kind="forward", B=1, Hq=32, Hkv=2, N=8192, d=64, window=256, sinks=16, type="bf16"),
        # long-context prompt pass at a 1024-token window
        dict(name="forward long", kind="forward", B=1, Hq=32, Hkv=8, N=32768, d=128, window=1024, sinks=64, type="bf16"),
        # a short odd batch in 32 bits, as in an evaluation
        dict(name="forward odd f32", kind="forward", B=2, Hq=4, Hkv=2, N=1021, d=64, window=200, sinks=4, type="f32"),
        # a training step's attention layer at 16K tokens
        dict(name="train long", kind="train", B=1, Hq=32, Hkv=8, N=16384, d=128, window=1024, sinks=64, type="bf16"),
        # fine-tuning batches of odd length
        dict(name="train odd", kind="train", B=2, Hq=16, Hkv=4, N=4099, d=64, window=512, sinks=1, type="bf16"),
        # gradient checks and small models in 32 bits
        dict(name="train f32", kind="train", B=1, Hq=8, Hkv=8, N=1000, d=128, window=128, sinks=16, type="f32"),
        # one token for each of 64 sequences
        dict(name="append tokens", kind="append", seqs=64, new=1, old=4000, Hq=32, Hkv=8, d=128, page=16, window=0, sinks=0, type="bf16"),
        # prompt chunks of a few sequences
        dict(name="append chunks", kind="append", seqs=8, new=2048, old=8192, Hq=32, Hkv=8, d=128, page=64, window=0, sinks=0, type="bf16"),
        # one token of one long conversation
        dict(name="attend one token", kind="attend", seqs=1, new=1, old=65535, Hq=32, Hkv=8, d=128, page=64, window=0, sinks=0, type="bf16"),
        # one token for each of 64 conversations of all lengths
        dict(name="attend tokens", kind="attend", seqs=64, new=1, old=8000, Hq=32, Hkv=8, d=128, page=16, window=0, sinks=0, type="bf16"),
        # chunked prefill: prompt chunks behind cached tokens
        dict(name="attend chunks", kind="attend", seqs=4, new=2048, old=14000, Hq=32, Hkv=8, d=128, page=64, window=0, sinks=0, type="bf16"),
        # a small model's chunks with a window, in 32 bits
        dict(name="attend window f32", kind="attend", seqs=5, new=301, old=3001, Hq=8, Hkv=2, d=64, page=32, window=1000, sinks=4, type="f32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["forward", "train", "append", "attend"])
    d = rng.choice([64, 128])
    kind_type = "f32" if rng.random() < 0.25 else "bf16"
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8] if Hkv < 8 else [1, 2, 4])
    sinks = rng.choice([0, 1, 4, 16, 64, rng.randint(2, 200)])
    if kind in ("forward", "train"):
        top = 2048 if kind_type == "f32" else 16384 if kind == "forward" else 8192
        N = _spread(rng, 1, top)
        window = _spread(rng, 16, 1024)
        if N <= 2048 and rng.random() < 0.2:
            window = EVERYTHING
        return dict(kind=kind, B=rng.choice([1, 2]), Hq=Hq, Hkv=Hkv, N=N, d=d, window=window, sinks=sinks, type=kind_type)
    page = rng.choice([16, 32, 64, 128, 256])
    window = 0 if rng.random() < 0.5 else _spread(rng, 16, 4096)
    if rng.random() < 0.5:
        seqs, new, old = _spread(rng, 1, 64), rng.choice([1, 1, 2, 5]), _spread(rng, 1, 8000)
    else:
        seqs, new, old = rng.randint(1, 4), _spread(rng, 16, 1500), _spread(rng, 1, 8000)
    if kind_type == "f32":
        seqs, new, old = min(seqs, 8), min(new, 500), min(old, 4000)
    return dict(kind=kind, seqs=seqs, new=new, old=old, Hq=Hq, Hkv=Hkv, d=d, page=page, window=window, sinks=sinks if window else 0, type=kind_type)


def _lengths(case):
    """New and cached tokens of each sequence. Several sequences are ragged: the i-th has between all and a quarter of them."""
    S = case["seqs"]
    share = [1.0 - 0.75 * ((i * 7) % S) / S for i in range(S)]
    new = [max(1, int(case["new"] * (s if case["new"] > 5 else 1.0))) for s in share]
    return new, [int(case["old"] * s) + n for s, n in zip(share, new)]


def _window(case):
    return case["window"] or EVERYTHING


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["type"]]

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)

    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    s = {"case": dict(case)}
    if case["kind"] in ("forward", "train"):
        B, N = case["B"], case["N"]
        s.update(Q=rand(B, Hq, N, d), K=rand(B, Hkv, N, d), V=rand(B, Hkv, N, d))
        if case["kind"] == "train":
            s["g"] = rand(B, Hq, N, d)
    else:
        new, total = _lengths(case)
        page, S, T = case["page"], case["seqs"], sum(new)
        need = [-(-n // page) for n in total]
        pool = sum(need) + 3
        order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((S, max(need)), -1, dtype=torch.int32)
        start, at = [0], 0
        order = order.cpu()
        for i in range(S):
            table[i, : need[i]] = order[at : at + need[i]]
            at += need[i]
            start.append(start[-1] + new[i])
        s.update(
            q_start=torch.tensor(start, dtype=torch.int32).cuda(),
            kv_len=torch.tensor(total, dtype=torch.int32).cuda(),
            table=table.cuda(), pool=pool, T=T, longest=max(total), most=max(new),
            Kc=rand(pool, page, Hkv, d), Vc=rand(pool, page, Hkv, d))
        if case["kind"] == "append":
            s.update(k=rand(T, Hkv, d), v=rand(T, Hkv, d))
        else:
            s.update(q=rand(T, Hq, d))
    s["own"] = {}
    return s


# ---------------------------------------------------------------- the framework's operators


def _own(s):
    from block_sparse_attention_ssa_b200 import api

    c, o = s["case"], s["own"]
    if c["kind"] in ("forward", "train"):
        if not o:
            o["dims"] = api.make_window_dims(c["B"], c["Hq"], c["Hkv"], c["N"], c["d"], c["window"], c["sinks"], c["type"])
            o["fwd"] = api.alloc_window_forward(o["dims"], s["Q"].device)
            if c["kind"] == "train":
                o["bwd"] = api.alloc_window_backward(o["dims"], s["Q"].device)
                o["ws"] = api.alloc_window_workspace(o["dims"], s["Q"].device)
        f = o["fwd"]
        api.ssa_fwd_window(o["dims"], s["Q"], s["K"], s["V"], f["h"], f["lse"])
        if c["kind"] == "forward":
            return f
        b = o["bwd"]
        api.ssa_bwd_window(o["dims"], s["Q"], s["K"], s["V"], f["h"], f["lse"], s["g"], b["dQ"], b["dK"], b["dV"], o["ws"])
        return {**f, **b}
    if not o:
        o["dims"] = api.make_paged_dims(c["seqs"], s["T"], c["Hq"], c["Hkv"], c["d"], c["page"], s["pool"], s["table"].shape[1],
                                        window=_window(c), sinks=c["sinks"], dtype=c["type"])
        if c["kind"] == "attend":
            o["out"] = api.alloc_paged(o["dims"], s["q"].device)
            o["ws"] = api.alloc_paged_workspace(o["dims"], s["q"].device)
    if c["kind"] == "append":
        api.ssa_paged_append(o["dims"], s["k"], s["v"], s["q_start"], s["kv_len"], s["table"], s["Kc"], s["Vc"])
        return {"K": s["Kc"], "V": s["Vc"]}
    r = o["out"]
    api.ssa_paged_attention(o["dims"], s["q"], s["Kc"], s["Vc"], s["q_start"], s["kv_len"], s["table"], r["h"], r["lse"], o["ws"])
    return r


# ---------------------------------------------------------------- the plain forms

BAND = 128  # queries that share one band of gathered keys


def _band(case, device):
    """For each block of BAND queries: the positions of the keys that some query of it sees, and which query sees which."""
    N, S = case["N"], min(case["sinks"], case["N"])
    nb = -(-N // BAND)
    reach = min(case["window"], nb * BAND)
    first = torch.arange(nb, device=device)[:, None] * BAND
    near = first - reach + torch.arange(reach + BAND, device=device)[None]
    far = torch.arange(S, device=device)[None].expand(nb, S)
    at = torch.cat([far, near], 1)
    t = (first + torch.arange(BAND, device=device)[None])[:, :, None]
    u = at[:, None, :]
    sees = (u >= 0) & (u <= t) & ((t - u < case["window"]) | (u < S)) & (t < N)
    again = torch.cat([torch.zeros_like(far, dtype=torch.bool), near < S], 1)  # a sink among the near keys counts once
    return nb, at.clamp(0, N - 1), sees & ~again[:, None, :]


def _blocks(x, nb, g):
    B, H, N, d = x.shape
    y = torch.zeros(B, H, nb * BAND, d, dtype=torch.float32, device=x.device)
    y[:, :, :N] = x
    return y.view(B, H // g, g, nb, BAND, d)


def _plain_window(s):
    c = s["case"]
    B, Hq, Hkv, N, d = c["B"], c["Hq"], c["Hkv"], c["N"], c["d"]
    g, scale, dt = Hq // Hkv, 1.0 / math.sqrt(d), s["Q"].dtype
    nb, at, sees = _band(c, s["Q"].device)
    Q = _blocks(s["Q"], nb, g)
    K, V = s["K"].float()[:, :, at], s["V"].float()[:, :, at]  # [B, Hkv, nb, keys, d]
    x = torch.einsum("bkgntd,bknud->bkgntu", Q, K) * scale
    x = x.masked_fill(~sees, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)  # the rows that fill the last block
    p = torch.exp(x - m)
    del x
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l == 0, torch.ones_like(l), l)
    h = torch.einsum("bkgntu,bknud->bkgntd", p, V)
    lse = (m + torch.log(l)).reshape(B, Hq, nb * BAND)[:, :, :N].contiguous()
    out = {"h": h.reshape(B, Hq, nb * BAND, d)[:, :, :N].to(dt), "lse": lse}
    if c["kind"] == "forward":
        return out
    G = _blocks(s["g"], nb, g)
    D = (G * h).sum(-1, keepdim=True)
    dx = (torch.einsum("bkgntd,bknud->bkgntu", G, V) - D) * p
    dQ = torch.einsum("bkgntu,bknud->bkgntd", dx, K) * scale
    dKb = torch.einsum("bkgntu,bkgntd->bknud", dx, Q) * scale
    dVb = torch.einsum("bkgntu,bkgntd->bknud", p, G)
    flat = at.reshape(-1)
    for name, band in (("dK", dKb), ("dV", dVb)):
        sums = torch.zeros(B, Hkv, N, d, dtype=torch.float32, device=Q.device)
        out[name] = sums.index_add_(2, flat, band.reshape(B, Hkv, -1, d)).to(dt)
    out["dQ"] = dQ.reshape(B, Hq, nb * BAND, d)[:, :, :N].to(dt)
    return out


def _rows(s):
    """Sequence and position of each packed new token."""
    c = s["case"]
    row = torch.arange(s["T"], device=s["table"].device, dtype=torch.int32)
    seq = torch.searchsorted(s["q_start"], row, right=True) - 1
    new = s["q_start"][seq + 1] - s["q_start"][seq]
    return seq, row - s["q_start"][seq], s["kv_len"][seq] - new + (row - s["q_start"][seq])


def _plain_append(s):
    page = s["case"]["page"]
    seq, _, pos = _rows(s)
    slot = s["table"][seq, (pos // page).long()].long()
    s["Kc"][slot, (pos % page).long()] = s["k"]
    s["Vc"][slot, (pos % page).long()] = s["v"]
    return {"K": s["Kc"], "V": s["Vc"]}


def _plain_attend(s):
    c = s["case"]
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    g, W, S = Hq // Hkv, _window(c), c["seqs"]
    seq, i, pos = _rows(s)
    i = i.long()
    Q = torch.zeros(S, s["most"], Hkv, g, d, device=s["q"].device)
    Q[seq, i] = s["q"].float().view(-1, Hkv, g, d)
    P = torch.full((S, s["most"]), -1, dtype=torch.int64, device=s["q"].device)
    P[seq, i] = pos.long()
    table = s["table"].clamp(min=0).long()
    K, V = (x[table].float().view(S, -1, Hkv, d) for x in (s["Kc"], s["Vc"]))
    u = torch.arange(K.shape[1], device=K.device)
    sees = (u <= P[:, :, None]) & ((P[:, :, None] - u < W) | (u < c["sinks"]))  # [S, most, keys]
    x = torch.einsum("sihgd,suhd->shgiu", Q, K) * (1.0 / math.sqrt(d))
    x.masked_fill_(~sees[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)  # the rows that fill the shorter chunks
    p = torch.exp(x - m)
    del x
    l = p.sum(-1, keepdim=True)
    h = torch.einsum("shgiu,suhd->sihgd", p, V) / torch.where(l == 0, torch.ones_like(l), l).permute(0, 3, 1, 2, 4)
    lse = (m + torch.log(l)).squeeze(-1).permute(0, 3, 1, 2)  # [S, most, Hkv, g]
    return {"h": h[seq, i].reshape(-1, Hq, d).to(s["q"].dtype), "lse": lse[seq, i].reshape(-1, Hq).t().contiguous()}


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    return _plain_append(state) if kind == "append" else _plain_attend(state) if kind == "attend" else _plain_window(state)


# ---------------------------------------------------------------- what a pass cannot do without


def _pairs(first, count, window, sinks):
    """Visible (query, key) pairs of `count` queries at positions first, first + 1, ..."""
    total = 0
    t0, t1 = first, first + count
    # below: everything; between: the window and part of the sinks; above: the window and the sinks
    a = min(t1, max(t0, window))
    total += (a * (a + 1) - t0 * (t0 + 1)) // 2
    b = min(t1, max(a, window + sinks))
    total += (b - a) * window + ((b - window) * (b - window + 1) - (a - window) * (a - window + 1)) // 2 if b > a else 0
    total += (t1 - b) * (window + sinks)
    return total


def work(case):
    es = 2 if case["type"] == "bf16" else 4
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["kind"] in ("forward", "train"):
        B, N = case["B"], case["N"]
        pairs = B * Hq * _pairs(0, N, case["window"], case["sinks"])
        q, k, rows = B * Hq * N * d * es, B * Hkv * N * d * es, 4 * B * Hq * N
        if case["kind"] == "forward":
            return {"bytes": 2 * q + 2 * k + rows, "flops": 4 * d * pairs}
        return {"bytes": 4 * q + 4 * k + rows, "flops": 14 * d * pairs}  # two products forward, five backward
    new, total = _lengths(case)
    T = sum(new)
    if case["kind"] == "append":
        return {"bytes": 4 * T * Hkv * d * es, "flops": 0}
    W = _window(case)
    pairs = sum(_pairs(n - c, c, W, case["sinks"]) for c, n in zip(new, total))
    seen = sum(n - max(0, n - c - W + 1 - min(case["sinks"], max(0, n - c - W + 1))) for c, n in zip(new, total))
    return {"bytes": 2 * T * Hq * d * es + 2 * seen * Hkv * d * es + 4 * T * Hq, "flops": 4 * d * Hq * pairs}


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_rows(Q, K, V, pos, W, S, scale):
    """One head: queries at positions pos over keys 0, 1, ...; [rows, d] each, in 64 bits."""
    u = torch.arange(K.shape[0], device=K.device)
    gap = pos[:, None] - u[None]
    x = torch.where((gap >= 0) & ((gap < W) | (u < S)[None]), (Q @ K.t()) * scale, -math.inf)
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    return p @ V, lse, p


def exact(case, seed):
    if case["kind"] == "append":
        return None
    s = prepare(case, seed)
    Hq, Hkv, d, W, S = case["Hq"], case["Hkv"], case["d"], _window(case), case["sinks"]
    g, scale, dev = Hq // Hkv, 1.0 / math.sqrt(d), "cuda"
    if case["kind"] == "attend":
        h = torch.zeros(s["T"], Hq, d, dtype=torch.float64, device=dev)
        lse = torch.zeros(Hq, s["T"], dtype=torch.float64, device=dev)
        new, total = _lengths(case)
        row = 0
        for b, (c, n) in enumerate(zip(new, total)):
            pages = s["table"][b, : -(-n // case["page"])].long()
            pos = torch.arange(n - c, n, device=dev)
            for k in range(Hkv):
                K, V = (x[pages, :, k].reshape(-1, d)[:n].double() for x in (s["Kc"], s["Vc"]))
                for q in range(k * g, k * g + g):
                    h[row : row + c, q], lse[q, row : row + c], _ = _exact_rows(s["q"][row : row + c, q].double(), K, V, pos, W, S, scale)
            row += c
        return {"h": h, "lse": lse}
    B, N = case["B"], case["N"]
    r = {"h": torch.zeros(B, Hq, N, d, dtype=torch.float64, device=dev), "lse": torch.zeros(B, Hq, N, dtype=torch.float64, device=dev)}
    if case["kind"] == "train":
        r.update({k: torch.zeros_like(s[k[1:]], dtype=torch.float64) for k in ("dQ", "dK", "dV")})
    step = 4096
    for b in range(B):
        for q in range(Hq):
            K, V = s["K"][b, q // g].double(), s["V"][b, q // g].double()
            for t0 in range(0, N, step):
                t1 = min(N, t0 + step)
                lo = max(0, t0 - W + 1)
                sel = torch.cat([torch.arange(min(S, lo), device=dev), torch.arange(lo, t1, device=dev)])
                pos = torch.arange(t0, t1, device=dev)
                gap = pos[:, None] - sel[None]
                Qt = s["Q"][b, q, t0:t1].double()
                x = torch.where((gap >= 0) & ((gap < W) | (sel < S)[None]), (Qt @ K[sel].t()) * scale, -math.inf)
                lse = torch.logsumexp(x, 1)
                p = torch.exp(x - lse[:, None])
                h = p @ V[sel]
                r["h"][b, q, t0:t1], r["lse"][b, q, t0:t1] = h, lse
                if case["kind"] == "train":
                    G = s["g"][b, q, t0:t1].double()
                    dx = p * (G @ V[sel].t() - (G * h).sum(1, keepdim=True))
                    r["dQ"][b, q, t0:t1] = dx @ K[sel] * scale
                    r["dK"][b, q // g].index_add_(0, sel, dx.t() @ Qt * scale)
                    r["dV"][b, q // g].index_add_(0, sel, p.t() @ G)
    return r
