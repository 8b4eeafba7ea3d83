"""Plain fp64 numpy forms of window attention with sinks and of attention over
a paged cache, one head and one dense matrix at a time, with the error bounds
that the tests hold the kernels to.

Visibility: query at position t sees key u when 0 <= u <= t and (t - u < window
or u < sinks).
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24  # half a step of fp32, relative
HALF_STEP = {"f32": U32, "bf16": 2.0 ** -8}


def visible(pos, n_keys: int, window: int, sinks: int) -> np.ndarray:
    t = np.asarray(pos, dtype=np.int64)[:, None]
    u = np.arange(n_keys, dtype=np.int64)[None]
    return (u <= t) & ((t - u < window) | (u < sinks))


def rows(Q, K, V, see, scale):
    """One head.  Returns h, lse, p and the largest scale * sum |q||k| of each row's visible keys;
    a row that sees nothing has h = 0, lse = -inf, p = 0."""
    Q, K, V = (np.asarray(x, dtype=np.float64) for x in (Q, K, V))
    x = np.where(see, (Q @ K.T) * scale, -np.inf)
    big = np.where(see, (np.abs(Q) @ np.abs(K).T) * scale, 0.0).max(axis=1, initial=0.0)
    m = x.max(axis=1, initial=-np.inf)
    ref = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(x - ref[:, None])
    s = e.sum(axis=1)
    some = s > 0
    p = e / np.where(some, s, 1.0)[:, None]
    lse = np.where(some, ref + np.log(np.where(some, s, 1.0)), -np.inf)
    return p @ V, lse, p, big


def weight_error(big, lse, n_keys: int, d: int):
    """Bound on the relative error of a weight exp(x - lse) formed in fp32: the d-term product (d + 2
    roundings of its terms), the scaled difference (two roundings of values up to |x| + |lse|), the
    exponential (2^-22) and, through lse, the sum of the row (n_keys roundings) and its logarithm."""
    lse = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    x = (d + 2) * U32 * big
    diff = 4 * U32 * (big + lse)
    return 2 * (x + diff) + (n_keys + 8) * U32 + 2 * 2.0 ** -22


def forward(Q, K, V, window, sinks, scale, dtype):
    """[B, Hq, N, d] over [B, Hkv, N, d]: h, lse and their tolerances, and each head's weights."""
    B, Hq, N, d = Q.shape
    g = Hq // K.shape[1]
    h, lse = np.zeros((B, Hq, N, d)), np.zeros((B, Hq, N))
    tol_h, tol_lse, werr = np.zeros_like(h), np.zeros_like(lse), np.zeros_like(lse)
    P = np.zeros((B, Hq, N, N))
    see = visible(np.arange(N), N, window, sinks)
    for b in range(B):
        for q in range(Hq):
            h[b, q], lse[b, q], P[b, q], big = rows(Q[b, q], K[b, q // g], V[b, q // g], see, scale)
            werr[b, q] = weight_error(big, lse[b, q], N, d)
            tol_h[b, q] = row_tolerance(P[b, q], V[b, q // g], h[b, q], werr[b, q], dtype)
            tol_lse[b, q] = werr[b, q] + 4 * U32 * np.abs(lse[b, q])
    return dict(h=h, lse=lse, tol_h=tol_h, tol_lse=tol_lse, werr=werr, P=P)


def row_tolerance(p, V, h, werr, dtype):
    """|h error|: the weights' error and, in bf16, their rounding before the product, on sum p |v|
    (n roundings of its fp32 sum too); the output's rounding on |h| plus that."""
    mass = p @ np.abs(np.asarray(V, dtype=np.float64))
    half = HALF_STEP[dtype]
    w = 2 * werr + (half if dtype == "bf16" else 0.0) + (p.shape[1] + 2) * U32
    inner = w[:, None] * mass
    return inner + half * (np.abs(h) + inner) + 1e-37


def backward(Q, K, V, g_out, f, window, sinks, scale, dtype):
    """Gradients of <g, h> and their tolerances; f is what forward() returned."""
    Q, K, V, G = (np.asarray(x, dtype=np.float64) for x in (Q, K, V, g_out))
    B, Hq, N, d = Q.shape
    grp, half = Hq // K.shape[1], HALF_STEP[dtype]
    r = dict(dQ=np.zeros_like(Q), dK=np.zeros_like(K), dV=np.zeros_like(V))
    tol = {k: np.zeros_like(v) for k, v in r.items()}
    n = N * grp + 2
    inner = half if dtype == "bf16" else 0.0  # rounding of p and dx before the products
    for b in range(B):
        for q in range(Hq):
            k = q // grp
            P, h = f["P"][b, q], f["h"][b, q]
            D = (G[b, q] * h).sum(1, keepdims=True)
            dP = G[b, q] @ V[b, k].T
            dx = P * (dP - D)
            aG, aV, aQ, aK = np.abs(G[b, q]), np.abs(V[b, k]), np.abs(Q[b, q]), np.abs(K[b, k])
            # D is formed from the rounded h; dP is a d-term product
            eD = (aG * (f["tol_h"][b, q] + (d + 2) * U32 * np.abs(h))).sum(1, keepdims=True)
            w = 2 * f["werr"][b, q][:, None] + 4 * U32
            edx = P * (eD + (d + 2) * U32 * (aG @ aV.T)) * (1 + w) + w * np.abs(dx)
            edx = edx + inner * (np.abs(dx) + edx)
            r["dQ"][b, q] = dx @ K[b, k] * scale
            tol["dQ"][b, q] = scale * ((edx + n * U32 * np.abs(dx)) @ aK)
            r["dK"][b, k] += dx.T @ Q[b, q] * scale
            tol["dK"][b, k] += scale * ((edx + n * U32 * np.abs(dx)).T @ aQ)
            r["dV"][b, k] += P.T @ G[b, q]
            tol["dV"][b, k] += ((w + inner + n * U32) * P).T @ aG
    for name in r:
        tol[name] += half * (np.abs(r[name]) + tol[name]) + 1e-37
    return r, tol


def gather(cache, table_row, length: int, page: int, head: int):
    """Keys 0..length-1 of one sequence and whether a page holds each ([pages, page, Hkv, d] cache)."""
    d = cache.shape[-1]
    out, held = np.zeros((length, d)), np.zeros(length, dtype=bool)
    for u in range(length):
        pg = int(table_row[u // page])
        if 0 <= pg < cache.shape[0]:
            out[u] = cache[pg, u % page, head]
            held[u] = True
    return out, held


def paged(q, Kc, Vc, q_start, kv_len, table, page, window, sinks, scale, dtype):
    """q [T, Hq, d]; returns h, lse, their tolerances and which packed rows a sequence owns."""
    T, Hq, d = q.shape
    g = Hq // Kc.shape[2]
    h, lse = np.zeros((T, Hq, d)), np.full((Hq, T), -np.inf)
    tol_h, tol_lse, own = np.zeros_like(h), np.zeros_like(lse), np.zeros(T, dtype=bool)
    for b in range(len(kv_len)):
        q0, n, L = int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        if n <= 0:
            continue
        own[q0:q0 + n] = True
        see0 = visible(np.arange(L - n, L), L, window, sinks)
        for k in range(Kc.shape[2]):
            K, held = gather(Kc, table[b], L, page, k)
            V, _ = gather(Vc, table[b], L, page, k)
            see = see0 & held[None]
            used = see.any(axis=0)
            K, V = np.where(used[:, None], K, 0.0), np.where(used[:, None], V, 0.0)  # unseen rows may hold anything
            for e in range(k * g, k * g + g):
                hh, ll, p, big = rows(q[q0:q0 + n, e], K, V, see, scale)
                w = weight_error(big, ll, L, d)
                h[q0:q0 + n, e], lse[e, q0:q0 + n] = hh, ll
                tol_h[q0:q0 + n, e] = row_tolerance(p, V, hh, w, dtype)
                tol_lse[e, q0:q0 + n] = w + 4 * U32 * np.where(np.isfinite(ll), np.abs(ll), 0.0)
    return dict(h=h, lse=lse, tol_h=tol_h, tol_lse=tol_lse, own=own)
