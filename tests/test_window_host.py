"""Window attention and the paged cache without a GPU: the 64-bit forms against
independent ones (dense loops, torch, differences), and the refusals of the C
ABI and of the Python binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_ssa_b200 import api
from oracle import window_oracle as W


@pytest.fixture(scope="module")
def lib():
    return api.load_library()


def _rand(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("N,window,sinks", [(1, 1, 0), (5, 1, 0), (7, 2, 3), (9, 4, 1), (9, 100, 0), (9, 3, 100)])
def test_forward_by_loops(N, window, sinks):
    Q, K, V = _rand(1, 1, 2, N, 4), _rand(2, 1, 1, N, 4), _rand(3, 1, 1, N, 4)
    f = W.forward(Q, K, V, window, sinks, 0.5, "f32")
    for q in range(2):
        for t in range(N):
            e = {u: math.exp(0.5 * float(Q[0, q, t] @ K[0, 0, u])) for u in range(N)
                 if u <= t and (u > t - window or u < sinks)}
            s = sum(e.values())
            np.testing.assert_allclose(f["h"][0, q, t], sum(e[u] * V[0, 0, u] for u in e) / s, rtol=1e-12)
            assert abs(f["lse"][0, q, t] - math.log(s)) < 1e-12


def test_everything_is_causal_attention():
    Q, K, V = (torch.from_numpy(_rand(i, 1, 3, 33, 8)) for i in range(3))
    f = W.forward(Q.numpy(), K.numpy(), V.numpy(), 33, 0, 1 / math.sqrt(8), "f32")
    ref = torch.nn.functional.scaled_dot_product_attention(Q, K, V, is_causal=True)
    np.testing.assert_allclose(f["h"], ref.numpy(), rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (50, 0)])
def test_backward_by_differences(window, sinks):
    B, Hq, Hkv, N, d = 1, 4, 2, 7, 3
    x = dict(Q=_rand(1, B, Hq, N, d), K=_rand(2, B, Hkv, N, d), V=_rand(3, B, Hkv, N, d))
    g = _rand(4, B, Hq, N, d)

    def loss(**y):
        return float((W.forward(y["Q"], y["K"], y["V"], window, sinks, 0.6, "f32")["h"] * g).sum())

    r, _ = W.backward(x["Q"], x["K"], x["V"], g, W.forward(**x, window=window, sinks=sinks, scale=0.6, dtype="f32"),
                      window, sinks, 0.6, "f32")
    for name in x:
        for i in np.random.default_rng(5).choice(x[name].size, 12, replace=False):
            up, down = dict(x), dict(x)
            up[name], down[name] = x[name].copy(), x[name].copy()
            up[name].flat[i] += 1e-5
            down[name].flat[i] -= 1e-5
            assert abs((loss(**up) - loss(**down)) / 2e-5 - r["d" + name].flat[i]) < 1e-7


def test_paged_is_the_contiguous_form():
    """A sequence's last rows over scattered pages are the same rows of the contiguous form; a missing
    page's positions do not count; a row at a negative position is empty."""
    rng = np.random.default_rng(0)
    Hq, Hkv, d, page, L, n = 4, 2, 8, 16, 45, 10
    K, V, Q = _rand(1, 1, Hkv, L, d), _rand(2, 1, Hkv, L, d), _rand(3, 1, Hq, L, d)
    Kc, Vc = _rand(4, 7, page, Hkv, d), _rand(5, 7, page, Hkv, d)
    table = rng.permutation(7)[:3][None].astype(np.int32)
    for u in range(L):
        Kc[table[0, u // page], u % page] = K[0, :, u]
        Vc[table[0, u // page], u % page] = V[0, :, u]
    f = W.forward(Q, K, V, 20, 3, 0.3, "f32")
    q = np.ascontiguousarray(Q[0, :, L - n:].transpose(1, 0, 2))
    r = W.paged(q, Kc, Vc, [0, n], [L], table, page, 20, 3, 0.3, "f32")
    np.testing.assert_allclose(r["h"].transpose(1, 0, 2), f["h"][0, :, L - n:], rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(r["lse"], f["lse"][0, :, L - n:], rtol=1e-12)
    short = W.paged(q, Kc, Vc, [0, n], [4], table, page, 20, 3, 0.3, "f32")
    assert np.all(short["h"][:6] == 0) and np.all(np.isneginf(short["lse"][:, :6])) and np.all(np.isfinite(short["lse"][:, 6:]))
    gone = W.paged(q, Kc, Vc, [0, n], [L], np.array([[-1, 7, -5]], dtype=np.int32), page, 20, 3, 0.3, "f32")
    assert np.all(gone["h"] == 0) and np.all(np.isneginf(gone["lse"]))


# ---------------------------------------------------------------- refusals

def _tensor(ptr=16, sb=4096 * 128, sh=4096 * 128, sn=128):
    return ctypes.pointer(api.ssa_tensor_t(ptr, sb, sh, sn))


def _p(x=256):
    return ctypes.c_void_p(x)


def _window_calls(lib, d, t=None, ws=1 << 50):
    t = t or _tensor()
    yield lib.ssa_fwd_window(ctypes.byref(d), t, t, t, t, _p(), None)
    yield lib.ssa_bwd_window(ctypes.byref(d), t, t, t, t, _p(), t, t, t, t, _p(), ws, None)


def _paged_calls(lib, d, t=None, ws=1 << 50):
    t = t or _tensor()
    yield lib.ssa_paged_append(ctypes.byref(d), t, t, _p(), _p(), _p(), t, t, None)
    yield lib.ssa_paged_attention(ctypes.byref(d), t, t, t, _p(), _p(), _p(), t, _p(), _p(), ws, None)


BAD = [("scale", 0.0), ("scale", -1.0), ("scale", float("inf")), ("scale", float("nan")), ("dtype", 2), ("dtype", -1),
       ("window", 0), ("window", -3), ("sinks", -1), ("Hq", -1), ("Hq", 5), ("Hkv", 0)]


@pytest.mark.parametrize("field,value", BAD + [("B", -1), ("N", -1)])
def test_window_bad_dims(lib, field, value):
    d = api.make_window_dims(1, 4, 2, 100, 64, 10, 2)
    setattr(d, field, value)
    assert set(_window_calls(lib, d)) == {api.SSA_ERR_INVALID_ARG}
    assert lib.ssa_window_workspace_bytes(ctypes.byref(d)) == 0


@pytest.mark.parametrize("field,value", [("d", 96), ("d", 0), ("N", (1 << 24) + 1), ("B", 40000)])
def test_window_unsupported_dims(lib, field, value):
    d = api.make_window_dims(1, 4, 2, 100, 64, 10, 2)
    setattr(d, field, value)
    assert set(_window_calls(lib, d)) == {api.SSA_ERR_UNSUPPORTED}


@pytest.mark.parametrize("field,value", BAD + [("num_seqs", -1), ("total_q", -1), ("num_pages", 0), ("max_pages", 0)])
def test_paged_bad_dims(lib, field, value):
    d = api.make_paged_dims(2, 10, 4, 2, 64, 16, 8, 4)
    setattr(d, field, value)
    assert set(_paged_calls(lib, d)) == {api.SSA_ERR_INVALID_ARG}
    assert lib.ssa_paged_workspace_bytes(ctypes.byref(d)) == 0


@pytest.mark.parametrize("field,value", [("d", 80), ("page", 8), ("page", 48), ("page", 512), ("Hq", 130), ("heads", 65536),
                                         ("max_pages", (1 << 26) + 1), ("total_q", (1 << 30) + 1)])
def test_paged_unsupported_dims(lib, field, value):
    d = api.make_paged_dims(2, 10, 4, 2, 64, 16, 8, 4)
    for name in ("Hq", "Hkv") if field == "heads" else (field,):
        setattr(d, name, value)
    assert set(_paged_calls(lib, d)) == {api.SSA_ERR_UNSUPPORTED}


def test_empty_calls_do_nothing(lib):
    for kw in (dict(B=0), dict(N=0), dict(Hq=0)):
        d = api.make_window_dims(**{**dict(B=1, Hq=4, Hkv=2, N=100, d=64, window=10), **kw})
        assert set(_window_calls(lib, d)) == {api.SSA_OK}
    for kw in (dict(num_seqs=0), dict(total_q=0), dict(Hq=0)):
        d = api.make_paged_dims(**{**dict(num_seqs=2, total_q=10, Hq=4, Hkv=2, d=64, page=16, num_pages=8, max_pages=4), **kw})
        assert set(_paged_calls(lib, d)) == {api.SSA_OK}


def test_bad_tensors(lib):
    w = api.make_window_dims(2, 4, 2, 100, 64, 10, 2)
    p = api.make_paged_dims(2, 10, 4, 2, 64, 16, 8, 4)
    for bad in (_tensor(ptr=8), _tensor(sn=100), _tensor(sn=32), _tensor(sb=-64), _tensor(sh=32), _tensor(ptr=0),
                _tensor(sn=1 << 40)):
        assert set(_window_calls(lib, w, bad)) == {api.SSA_ERR_INVALID_ARG}
        assert set(_paged_calls(lib, p, bad)) == {api.SSA_ERR_INVALID_ARG}
    good, flat = _tensor(), _tensor(sh=0)
    # heads laid over one another: fine to read, refused where they would be written
    assert lib.ssa_fwd_window(ctypes.byref(w), good, good, good, flat, _p(), None) == api.SSA_ERR_INVALID_ARG
    assert lib.ssa_bwd_window(ctypes.byref(w), good, good, good, good, _p(), good, good, flat, good, _p(), 1 << 50,
                              None) == api.SSA_ERR_INVALID_ARG
    assert lib.ssa_paged_append(ctypes.byref(p), good, good, _p(), _p(), _p(), flat, good, None) == api.SSA_ERR_INVALID_ARG
    for i in range(5):
        ptrs = [_p()] * 5
        ptrs[i] = None
        got = lib.ssa_paged_attention(ctypes.byref(p), good, good, good, ptrs[0], ptrs[1], ptrs[2], good, ptrs[3], ptrs[4],
                                      1 << 50, None)
        assert got == (api.SSA_ERR_WORKSPACE if i == 4 else api.SSA_ERR_INVALID_ARG)
    assert lib.ssa_fwd_window(ctypes.byref(w), good, good, good, good, None, None) == api.SSA_ERR_INVALID_ARG
    assert lib.ssa_fwd_window(None, good, good, good, good, _p(), None) == api.SSA_ERR_INVALID_ARG
    assert lib.ssa_paged_append(None, good, good, _p(), _p(), _p(), good, good, None) == api.SSA_ERR_INVALID_ARG


def test_workspaces(lib):
    w = api.make_window_dims(1, 4, 2, 100, 64, 10, 2)
    p = api.make_paged_dims(2, 10, 4, 2, 64, 16, 8, 4)
    t = _tensor()
    for need, call in ((api.ssa_window_workspace_bytes(w),
                        lambda ws, n: lib.ssa_bwd_window(ctypes.byref(w), t, t, t, t, _p(), t, t, t, t, ws, n, None)),
                       (api.ssa_paged_workspace_bytes(p),
                        lambda ws, n: lib.ssa_paged_attention(ctypes.byref(p), t, t, t, _p(), _p(), _p(), t, _p(), ws, n, None))):
        assert need > 0 and need % 256 == 0
        assert call(_p(), need - 1) == api.SSA_ERR_WORKSPACE
        assert call(None, need) == api.SSA_ERR_WORKSPACE
        assert call(_p(128), need) == api.SSA_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hkv", [(1, 1, 1), (1, 37, 1), (1, 148, 1), (1, 4096, 8), (64, 64, 64)])
def test_workspace_of_the_longest_sequences(lib, B, Hq, Hkv, dtype):
    """2^24 tokens, everything visible: -lse and -D, and partials of tiles that are cut, each into chunks of an equal
    share (a 296th of the steps, 2^30 at most): no more tiles than shares, and a chunk begun for each."""
    N, d, tile = 1 << 24, 128, 128 if dtype == "bf16" else 64
    need = api.ssa_window_workspace_bytes(api.make_window_dims(B, Hq, Hkv, N, d, dtype=dtype))
    rows = 2 * B * Hq * N * 4
    steps = B * Hq * (N // tile) * (N // tile + 1) // 2
    partials = 2 * max(296, -(-steps >> 30))
    assert rows <= need <= rows + partials * 2 * tile * d * 4 + 1024


def test_binding_refuses_wrong_tensors():
    d = api.make_window_dims(1, 4, 2, 10, 64, 5, 1, "f32")
    q, k, lse = torch.zeros(1, 4, 10, 64), torch.zeros(1, 2, 10, 64), torch.zeros(1, 4, 10)
    with pytest.raises(ValueError, match="CUDA"):
        api.ssa_fwd_window(d, q, k, k, q, lse)
    with pytest.raises(ValueError, match="Q"):
        api.ssa_fwd_window(d, q.bfloat16(), k, k, q, lse)
    with pytest.raises(ValueError, match="Q"):
        api.ssa_fwd_window(d, q[:, :, :9], k, k, q, lse)
    p = api.make_paged_dims(1, 3, 4, 2, 64, 16, 5, 2, dtype="f32")
    with pytest.raises(ValueError):
        api.ssa_paged_append(p, torch.zeros(3, 2, 64), torch.zeros(3, 2, 64), torch.zeros(2, dtype=torch.int32),
                             torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32),
                             torch.zeros(5, 16, 2, 64), torch.zeros(5, 16, 2, 64))


def _bwd_dq(lib, dq, B=2, Hq=4, N=100):
    """The answer to a workspace that is too small, once the tensors are taken: nothing is enqueued."""
    w, t, good = api.make_window_dims(B, Hq, Hq, N, 64, 10), _tensor(), _tensor(16, 1 << 30, 1 << 25, 64)
    return lib.ssa_bwd_window(ctypes.byref(w), t, t, t, t, _p(), t, dq, good, good, _p(), 0, None)


# [B, H, N, 64] with B = 2, H = 4, N = 100: strides whose slices meet
MEETING = {
    "heads_and_rows": (4 * 6400, 64, 64), "half_a_head": (4 * 6400, 128, 64), "batches_and_heads": (6400, 6400, 64),
    "last_row": (4 * 6400, 6400 - 64, 64), "batch_in_the_last_head": (4 * 6400 - 8, 6400, 64), "rows_over_heads": (25600, 64, 192),
    "rows_over_batches": (256, 64, 256), "far_rows": (64, 1 << 26, 1 << 20),
}
APART = {
    "heads_first": (4 * 6400, 6400, 64), "rows_first": (4 * 6400, 64, 256), "padded": (32000, 7400, 72), "batches_inside": (64, 128, 512),
    "other_rows": (128, 25600, 256), "far": (1 << 37, 1 << 35, 1 << 28),
}


def test_outputs_that_lie_over_themselves(lib):
    for name, s in MEETING.items():
        bad = _tensor(16, *s)
        w, t, good = api.make_window_dims(2, 4, 4, 100, 64, 10), _tensor(), _tensor(16, 25600, 6400, 64)
        assert lib.ssa_fwd_window(ctypes.byref(w), t, t, t, bad, _p(), None) == api.SSA_ERR_INVALID_ARG, name
        assert _bwd_dq(lib, bad) == api.SSA_ERR_INVALID_ARG, name
        for i in range(3):
            grads = [good] * 3
            grads[i] = bad
            assert lib.ssa_bwd_window(ctypes.byref(w), t, t, t, t, _p(), t, *grads, _p(), 1 << 50, None) == api.SSA_ERR_INVALID_ARG
        p = api.make_paged_dims(1, 100, 4, 4, 64, 128, 2, 4)
        for cache in ((bad, good), (good, bad)):  # a page has 128 rows
            assert lib.ssa_paged_append(ctypes.byref(p), t, t, _p(), _p(), _p(), *cache, None) == api.SSA_ERR_INVALID_ARG
        if name not in ("batches_and_heads", "batch_in_the_last_head", "rows_over_batches"):  # no batches there
            assert lib.ssa_paged_attention(ctypes.byref(p), t, t, t, _p(), _p(), _p(), bad, _p(), _p(), 1 << 50,
                                           None) == api.SSA_ERR_INVALID_ARG, name
    for name, s in APART.items():
        assert _bwd_dq(lib, _tensor(16, *s)) == api.SSA_ERR_WORKSPACE, name
    # a dimension of length one has no slices to meet
    assert _bwd_dq(lib, _tensor(16, 64, 64, 64), B=1, Hq=2, N=1) == api.SSA_ERR_WORKSPACE
    assert _bwd_dq(lib, _tensor(16, 64, 64, 64), B=1, Hq=1) == api.SSA_ERR_WORKSPACE
