"""NaN and infinities in the window and paged calls: a value reaches the rows
whose mask leaves it, and no others.  Wanted are sums in 64 bits over the
visible pairs alone; the bounds are those of oracle/window_oracle.py at the same
inputs with zeros in place of what is not finite."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_ssa_b200 import api
from oracle import window_oracle as W
from tests.gpu_util import ensure_library, f64
from tests.test_gpu_paged import Batch
from tests.test_gpu_window import _inputs, _run

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")

# B, Hq, Hkv, N, d, window, sinks
SHAPES = {
    "one_slot": (1, 4, 2, 400, 64, 90, 5),
    "one_slot_d128": (2, 3, 1, 333, 128, 200, 1),
    "everything": (1, 6, 2, 300, 128, api.EVERYTHING, 0),
    # enough heads for two 128-row tiles at once
    "two_slots": (1, 64, 8, 600, 64, 130, 70),
    "two_slots_d128": (1, 75, 15, 500, 128, 129, 3),
}


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


def _sum(weights, see, x):
    """Row t: the sum of weights[t, u] x[u] over the u it sees."""
    out = np.zeros((len(weights), x.shape[1]))
    for t in range(len(weights)):
        out[t] = weights[t, see[t]] @ x[see[t]]
    return out


def _head(Q, K, V, see, scale):
    x = np.where(see, (Q @ K.T) * scale, -INF)
    some = see.any(axis=1)
    m = np.where(some, np.max(x, axis=1), 0.0)  # NaN where one is seen
    m = np.where(m == -INF, 0.0, m)
    e = np.where(see, np.exp(x - m[:, None]), 0.0)
    s = e.sum(axis=1)
    p = e / np.where(some, s, 1.0)[:, None]
    return _sum(p, see, V), np.where(some, m + np.log(np.where(some, s, 1.0)), -INF), p


def _same(name, got, want, tol):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), (name, np.argwhere(np.isnan(got) != np.isnan(want))[:5])
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), name
    off = np.where(fine, np.abs(np.where(fine, got, 0.0) - np.where(fine, want, 0.0)) - tol, -1.0)
    assert off.max(initial=-1.0) <= 0, (name, np.unravel_index(off.argmax(), off.shape), off.max())


def _window_case(name, dtype, spoil, train):
    B, Hq, Hkv, N, d, window, sinks = SHAPES[name]
    scale, grp = 1 / math.sqrt(d), Hq // Hkv
    host = _inputs(B, Hq, Hkv, N, d, dtype, 17)
    for k, at, value in spoil(N):
        host[k][(0,) + at] = value
    dims = api.make_window_dims(B, Hq, Hkv, N, d, window, sinks, dtype)
    got = _run(dims, {k: v.cuda() for k, v in host.items()}, train)
    x = {k: v.double().numpy() for k, v in host.items()}
    clean = {k: np.where(np.isfinite(v), v, 0.0) for k, v in x.items()}
    f = W.forward(clean["Q"], clean["K"], clean["V"], window, sinks, scale, dtype)
    see = W.visible(np.arange(N), N, window, sinks)
    h, lse = np.zeros((B, Hq, N, d)), np.zeros((B, Hq, N))
    dQ, dK, dV = np.zeros_like(x["Q"]), np.zeros_like(x["K"]), np.zeros_like(x["V"])
    with np.errstate(all="ignore"):
        for b in range(B):
            for q in range(Hq):
                Q, K, V, G = x["Q"][b, q], x["K"][b, q // grp], x["V"][b, q // grp], x["g"][b, q]
                h[b, q], lse[b, q], p = _head(Q, K, V, see, scale)
                if train:
                    dx = np.where(see, p * (G @ V.T - (G * h[b, q]).sum(1, keepdims=True)), 0.0)
                    dQ[b, q] = _sum(dx, see, K) * scale
                    dK[b, q // grp] += _sum(dx.T, see.T, Q) * scale
                    dV[b, q // grp] += _sum(p.T, see.T, G)
    _same("h", got["h"], h, f["tol_h"])
    _same("lse", got["lse"], lse, f["tol_lse"])
    if train:
        _, tol = W.backward(clean["Q"], clean["K"], clean["V"], clean["g"], f, window, sinks, scale, dtype)
        for k, want in (("dQ", dQ), ("dK", dK), ("dV", dV)):
            _same(k, got[k], want, tol[k])


# (tensor, index behind the batch, value)
FORWARD = {
    # behind the tokens that use them, as the rows that fill a padded batch
    "tail": lambda N: [("V", (slice(None), slice(N - 3, None)), NAN), ("K", (slice(None), slice(N - 2, None)), NAN)],
    # behind the sinks in a tile that every later token loads
    "behind_the_sinks": lambda N: [("V", (0, 100), NAN), ("V", (slice(None), 71, 5), INF)],
    "one_element": lambda N: [("V", (0, 200, 33), INF), ("V", (0, 203, 2), -INF), ("V", (0, 210, 2), INF), ("V", (0, 131, 60), NAN)],
    # a sink that far tokens meet alone in their first tile: its NaN comes before the first finite logit
    "first_sink": lambda N: [("K", (0, 0), NAN)],
    "a_key_and_a_query": lambda N: [("K", (0, 150), NAN), ("Q", (1, 160), NAN), ("V", (0, 0), NAN)],
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what", list(FORWARD))
@pytest.mark.parametrize("name", list(SHAPES))
def test_window_forward(name, what, dtype):
    _window_case(name, dtype, FORWARD[what], train=False)


# fp32 alone: infinities and the largest magnitudes where tokens see them; -infinity in a key (finite logits of its other
# values) hides the key from queries that are positive there
FP32 = {
    "infinities": lambda N: [("V", (0, 20), INF), ("V", (slice(None), 190, 7), -INF), ("V", (0, 191, 7), INF)],
    "largest": lambda N: [("V", (0, 40, slice(0, 8)), 3.4028e38), ("V", (slice(None), 201), -3.4027e38)],
    "hiding_keys": lambda N: [("K", (slice(None), 50, 0), -INF), ("K", (0, 180, 0), -INF)],
}


@pytest.mark.parametrize("what", list(FP32))
@pytest.mark.parametrize("name", list(SHAPES))
def test_window_forward_fp32(name, what):
    _window_case(name, "f32", FP32[what], train=False)


BACKWARD = {
    # rows that fill a padded batch, with gradients and without
    "tail": lambda N: [("V", (slice(None), slice(N - 3, None)), NAN), ("K", (slice(None), slice(N - 2, None)), NAN),
                       ("Q", (slice(None), slice(N - 2, None)), NAN), ("g", (slice(None), slice(N - 3, None)), NAN)],
    "tail_of_inputs": lambda N: [("K", (slice(None), slice(N - 2, None)), NAN), ("Q", (slice(None), slice(N - 1, None)), NAN)],
    # a key behind the sinks, a late token whose gradient the sinks get
    "behind_the_sinks": lambda N: [("K", (0, 100), NAN), ("g", (1, N - 40), NAN)],
    "a_late_query": lambda N: [("Q", (0, N - 70), NAN)],
    "one_element": lambda N: [("K", (0, 131, 7), NAN), ("g", (0, 210, 3), INF), ("g", (2, 140, 9), NAN)],
    "a_value": lambda N: [("V", (0, 150, 20), NAN)],
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what", list(BACKWARD))
@pytest.mark.parametrize("name", list(SHAPES))
def test_window_backward(name, what, dtype):
    _window_case(name, dtype, BACKWARD[what], train=True)


# new tokens, tokens in all, Hq, Hkv, d, page; then V rows that are spoiled: (sequence, position)
PAGED = {
    "chunks": (([70, 1, 129, 5], [500, 33, 129, 1111], 8, 2, 128, 16), [(0, 450), (0, 499), (2, 60), (3, 1107), (3, 300)]),
    "cut_chunk": (([300], [2400], 4, 1, 64, 64), [(0, 2150), (0, 2399), (0, 900)]),
    # rows at negative positions beside rows that see NaN
    "empty_rows": (([10, 5, 70], [4, 0, 66], 4, 2, 64, 16), [(0, 2), (0, 3), (2, 0), (2, 60)]),
    "tokens": (([1, 1, 4], [700, 900, 130], 8, 2, 64, 32), [(0, 650), (2, 127), (2, 129), (1, 5)]),
}


@pytest.mark.parametrize("window,sinks", [(None, 0), (200, 20)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(PAGED))
def test_paged(name, dtype, window, sinks):
    args, bad = PAGED[name]
    b = Batch(*args, dtype)
    for i, (s, u) in enumerate(bad):
        row = b.caches[1][b.table[s, u // b.page], u % b.page]
        if i % 2:
            row[0, 5] = INF
        else:
            row[:] = NAN
    got = b.attend(window, sinks)
    Kc, Vc = (np.nan_to_num(c.double().numpy(), posinf=0.0) for c in b.caches)
    w = api.EVERYTHING if window is None else window
    r = W.paged(b.q.double().numpy(), Kc, Vc, b.q_start.numpy(), b.kv_len.numpy(), b.table.numpy(), b.page, w, sinks,
                1 / math.sqrt(b.d), dtype)
    h, lse = r["h"].copy(), r["lse"].copy()
    for i, (s, u) in enumerate(bad):
        q0, n, L = int(b.q_start[s]), b.new[s], b.total[s]
        see = W.visible(np.arange(L - n, L), L, w, sinks)[:, u]
        heads = slice(0, b.Hq // b.Hkv) if i % 2 else slice(None)
        cols = slice(5, 6) if i % 2 else slice(None)
        block = h[q0:q0 + n][see]  # copies: sums of what was there and the spoiled value
        block[:, heads, cols] += INF if i % 2 else NAN
        h[q0:q0 + n][see] = block
    own = r["own"]
    _same("h", f64(got["h"])[own], h[own], r["tol_h"][own])
    _same("lse", f64(got["lse"])[:, own], lse[:, own], r["tol_lse"][:, own])
    assert np.all(f64(got["h"])[~own] == 5.0)
