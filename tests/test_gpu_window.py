"""GPU parity of ssa_fwd_window and ssa_bwd_window with the 64-bit form, each
element within the bound that oracle/window_oracle.py derives for it."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_ssa_b200 import api
from oracle import window_oracle as W
from tests.gpu_util import ensure_library, f64, rel_l2

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EVERYTHING = api.EVERYTHING

# B, Hq, Hkv, N, d, window, sinks
SHAPES = {
    "one_token": (1, 1, 1, 1, 64, 1, 0),
    "one_token_gqa": (2, 6, 2, 1, 128, 5, 3),
    "two_tokens": (1, 2, 1, 2, 64, 1, 0),
    "self_only": (1, 2, 2, 130, 64, 1, 0),
    "self_and_sinks": (1, 4, 2, 200, 128, 1, 5),
    "below_tile": (2, 4, 1, 63, 64, 10, 2),
    "tile": (1, 4, 4, 128, 128, 64, 1),
    "past_tile": (1, 3, 1, 129, 64, 40, 0),
    "window_of_a_tile": (1, 4, 2, 515, 128, 128, 0),
    "odd_everything": (2, 6, 2, 517, 64, 101, 7),
    "many_sinks": (1, 4, 1, 600, 128, 65, 200),
    "sinks_reach_the_window": (1, 2, 1, 400, 64, 150, 300),
    "all_sinks": (1, 2, 1, 300, 128, 3, 1000),
    "everything": (1, 4, 2, 385, 64, EVERYTHING, 0),
    "everything_d128": (1, 8, 1, 450, 128, EVERYTHING, 9),
    "three_to_one": (1, 3, 1, 700, 128, 256, 16),
    "group_of_sixteen": (1, 16, 1, 257, 64, 70, 4),
    # enough heads for the form that holds two 128-row tiles at once
    "two_tiles": (1, 64, 8, 600, 64, 130, 70),
    "two_tiles_everything": (1, 50, 10, 641, 128, EVERYTHING, 0),
    "two_tiles_second_short": (1, 150, 50, 140, 64, 33, 3),
    "two_tiles_narrow": (2, 40, 8, 450, 128, 1, 1),
    # key tiles cut into chunks
    "cut_tiles": (1, 8, 1, 1400, 64, 65, 64),
}


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


def _inputs(B, Hq, Hkv, N, d, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda h: torch.randn(B, h, N, d, generator=gen).to(TYPES[dtype])  # noqa: E731
    return dict(Q=mk(Hq), K=mk(Hkv), V=mk(Hkv), g=mk(Hq))


def _nan(x):
    return torch.full_like(x, float("nan"))


def _run(dims, dev, train=True):
    out = {k: _nan(v) for k, v in api.alloc_window_forward(dims).items()}
    api.ssa_fwd_window(dims, dev["Q"], dev["K"], dev["V"], out["h"], out["lse"])
    if train:
        grads = {k: _nan(v) for k, v in api.alloc_window_backward(dims).items()}
        ws = api.alloc_window_workspace(dims).fill_(255)
        api.ssa_bwd_window(dims, dev["Q"], dev["K"], dev["V"], out["h"], out["lse"], dev["g"], grads["dQ"], grads["dK"],
                           grads["dV"], ws)
        out.update(grads)
    torch.cuda.synchronize()
    assert api.ssa_device_status() == api.SSA_OK
    return out


def within(name, got, want, tol):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fine), name
    assert np.array_equal(got[~fine], want[~fine]), name
    off = np.abs(np.where(fine, got, 0.0) - np.where(fine, want, 0.0)) - tol
    assert off.max(initial=-1.0) <= 0, (name, np.unravel_index(off.argmax(), off.shape), off.max())


def _check(out, host, window, sinks, scale, dtype, train=True):
    x = {k: v.double().numpy() for k, v in host.items()}
    f = W.forward(x["Q"], x["K"], x["V"], window, sinks, scale, dtype)
    within("h", out["h"], f["h"], f["tol_h"])
    within("lse", out["lse"], f["lse"], f["tol_lse"])
    if train:
        r, tol = W.backward(x["Q"], x["K"], x["V"], x["g"], f, window, sinks, scale, dtype)
        for k in r:
            within(k, out[k], r[k], tol[k])
            if np.linalg.norm(r[k]) > 1e-6 * np.linalg.norm(x["g"]):
                # the elements' roundings are independent: their norm is far inside the sum of bounds
                assert rel_l2(f64(out[k]), r[k]) < (1e-2 if dtype == "bf16" else 2e-5), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_forward_and_backward(name, dtype):
    B, Hq, Hkv, N, d, window, sinks = SHAPES[name]
    host = _inputs(B, Hq, Hkv, N, d, dtype, 11)
    dims = api.make_window_dims(B, Hq, Hkv, N, d, window, sinks, dtype)
    out = _run(dims, {k: v.cuda() for k, v in host.items()})
    _check(out, host, window, sinks, 1 / math.sqrt(d), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_and_broadcast_inputs(dtype):
    """[B, N, H, d] memory, keys and values shared by all heads and batches through zero strides, an upstream
    gradient shared by all heads, outputs written into slices of larger buffers that keep what lies around them."""
    B, H, N, d, window, sinks = 2, 4, 150, 64, 33, 2
    host = _inputs(B, H, 1, N, d, dtype, 5)
    host["K"], host["V"] = (host[k][:1].expand(B, H, N, d) for k in ("K", "V"))
    host["g"] = host["g"][:, :1].expand(B, H, N, d)
    dims = api.make_window_dims(B, H, H, N, d, window, sinks, dtype, scale=0.2)
    dev = dict(Q=host["Q"].cuda().transpose(1, 2).contiguous().transpose(1, 2),
               K=host["K"][:1, :1].cuda().expand(B, H, N, d), V=host["V"][:1, :1].cuda().expand(B, H, N, d),
               g=host["g"][:, :1].cuda().expand(B, H, N, d))
    big = {k: torch.full((B, N + 2, H + 1, d + 8), 7.0, dtype=TYPES[dtype], device="cuda") for k in ("h", "dQ", "dK", "dV")}
    out = {k: v[:, 1:-1, :H, :d].transpose(1, 2) for k, v in big.items()}
    out["lse"] = torch.empty(B, H, N, device="cuda")
    ws = api.alloc_window_workspace(dims)
    api.ssa_fwd_window(dims, dev["Q"], dev["K"], dev["V"], out["h"], out["lse"])
    api.ssa_bwd_window(dims, dev["Q"], dev["K"], dev["V"], out["h"], out["lse"], dev["g"], out["dQ"], out["dK"], out["dV"], ws)
    torch.cuda.synchronize()
    _check(out, host, window, sinks, 0.2, dtype)
    for v in big.values():
        v[:, 1:-1, :H, :d] = 7.0
        assert bool((v == 7.0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_logits_and_far_offsets(dtype):
    """Logits of some hundreds, whose running maxima grow along a row, and a value far from zero."""
    B, Hq, Hkv, N, d, window, sinks = 1, 2, 1, 400, 64, 300, 3
    host = _inputs(B, Hq, Hkv, N, d, dtype, 3)
    ramp = torch.linspace(0.1, 12.0, N)[None, None, :, None]
    host["Q"] = host["Q"].abs().to(TYPES[dtype])
    host["K"] = (host["K"].float().abs() * ramp).to(TYPES[dtype])
    host["V"] = (host["V"].float() + 100.0).to(TYPES[dtype])
    dims = api.make_window_dims(B, Hq, Hkv, N, d, window, sinks, dtype)
    out = _run(dims, {k: v.cuda() for k, v in host.items()}, train=False)
    _check(out, host, window, sinks, 1 / math.sqrt(d), dtype, train=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_by_differences(dtype):
    """<g, h> along a random direction, by central differences of the 64-bit form at the kernel's inputs."""
    B, Hq, Hkv, N, d, window, sinks = 1, 4, 2, 140, 64, 50, 3
    host = _inputs(B, Hq, Hkv, N, d, dtype, 21)
    dims = api.make_window_dims(B, Hq, Hkv, N, d, window, sinks, dtype)
    out = _run(dims, {k: v.cuda() for k, v in host.items()})
    x = {k: v.double().numpy() for k, v in host.items()}
    rng = np.random.default_rng(2)
    f = W.forward(x["Q"], x["K"], x["V"], window, sinks, 1 / math.sqrt(d), dtype)
    _, tol = W.backward(x["Q"], x["K"], x["V"], x["g"], f, window, sinks, 1 / math.sqrt(d), dtype)
    for k in ("Q", "K", "V"):
        way = rng.standard_normal(x[k].shape)
        val = []
        for e in (1e-5, -1e-5):
            y = {**x, k: x[k] + e * way}
            val.append((W.forward(y["Q"], y["K"], y["V"], window, sinks, 1 / math.sqrt(d), dtype)["h"] * x["g"]).sum())
        slope = (val[0] - val[1]) / 2e-5
        assert abs((f64(out["d" + k]) * way).sum() - slope) <= (tol["d" + k] * np.abs(way)).sum() + 1e-5 * abs(slope)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_calls_at_once(dtype):
    """Training steps of two shapes on two streams, each with its own workspace, many times over; then both in one
    graph, one after the other over one workspace."""
    shapes = [(1, 4, 2, 900, 128, 150, 20), (2, 2, 1, 333, 64, 1 << 20, 0)]
    state = []
    for i, s in enumerate(shapes):
        dims, x = api.make_window_dims(*s, dtype), {k: v.cuda() for k, v in _inputs(*s[:5], dtype, i).items()}
        state.append((dims, x, _run(dims, x), {**api.alloc_window_forward(dims), **api.alloc_window_backward(dims)},
                      api.alloc_window_workspace(dims)))

    def step(dims, x, out, ws, stream=None):
        api.ssa_fwd_window(dims, x["Q"], x["K"], x["V"], out["h"], out["lse"], stream=stream)
        api.ssa_bwd_window(dims, x["Q"], x["K"], x["V"], out["h"], out["lse"], x["g"], out["dQ"], out["dK"], out["dV"], ws,
                           stream=stream)

    def compare():
        torch.cuda.synchronize()
        assert api.ssa_device_status() == api.SSA_OK
        for _, _, want, out, _ in state:
            for k in out:
                assert torch.equal(out[k], want[k]), k
                out[k].fill_(3.0)

    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in state]
    for _ in range(10):
        for s, (dims, x, _, out, ws) in zip(streams, state):
            step(dims, x, out, ws, s)
    compare()
    shared = max((st[4] for st in state), key=torch.numel)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for dims, x, _, out, _ in state:
            step(dims, x, out, shared)
    for _ in range(3):
        graph.replay()
    compare()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_and_captured(dtype):
    """The same inputs give the same bits, eagerly, on another stream and from a captured graph with new inputs."""
    B, Hq, Hkv, N, d, window, sinks = 1, 4, 2, 1100, 128, 150, 20
    dims = api.make_window_dims(B, Hq, Hkv, N, d, window, sinks, dtype)
    first = {k: v.cuda() for k, v in _inputs(B, Hq, Hkv, N, d, dtype, 1).items()}
    second = {k: v.cuda() for k, v in _inputs(B, Hq, Hkv, N, d, dtype, 2).items()}
    want = [_run(dims, x) for x in (first, second)]
    again = _run(dims, first)
    for k in again:
        assert torch.equal(again[k], want[0][k]), k
    live = {k: v.clone() for k, v in first.items()}
    out = {**api.alloc_window_forward(dims), **api.alloc_window_backward(dims)}
    ws = api.alloc_window_workspace(dims)

    def step():
        api.ssa_fwd_window(dims, live["Q"], live["K"], live["V"], out["h"], out["lse"])
        api.ssa_bwd_window(dims, live["Q"], live["K"], live["V"], out["h"], out["lse"], live["g"], out["dQ"], out["dK"],
                           out["dV"], ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    for k in out:
        assert torch.equal(out[k], want[0][k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k, v in second.items():
        live[k].copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    for k in out:
        assert torch.equal(out[k], want[1][k]), k


def test_long_rows_against_a_sample():
    """A long sequence in bf16, checked on the rows and keys around tile and window borders."""
    B, Hq, Hkv, N, d, window, sinks = 1, 4, 2, 20011, 128, 1024, 64
    gen = torch.Generator(device="cuda").manual_seed(4)
    mk = lambda h: torch.randn(B, h, N, d, generator=gen, device="cuda").bfloat16()  # noqa: E731
    dev = dict(Q=mk(Hq), K=mk(Hkv), V=mk(Hkv), g=mk(Hq))
    dims = api.make_window_dims(B, Hq, Hkv, N, d, window, sinks, "bf16")
    out = _run(dims, dev)
    scale = 1 / math.sqrt(d)
    rows = torch.tensor([0, 1, 63, 64, 127, 128, 1023, 1024, 1087, 1088, 1089, 9999, 12800, 20009, 20010], device="cuda")
    u = torch.arange(N, device="cuda")
    see = lambda t: (u[None] <= t[:, None]) & ((t[:, None] - u[None] < window) | (u[None] < sinks))  # noqa: E731
    for q in range(Hq):
        Q, g = dev["Q"][0, q].double(), dev["g"][0, q].double()
        K, V = dev["K"][0, q // 2].double(), dev["V"][0, q // 2].double()
        x = torch.where(see(rows), Q[rows] @ K.t() * scale, -math.inf)
        lse = torch.logsumexp(x, 1)
        p = torch.exp(x - lse[:, None])
        h = p @ V
        assert float((out["h"][0, q, rows].double() - h).norm() / h.norm()) < 4e-3
        assert float((out["lse"][0, q, rows].double() - lse).abs().max()) < 1e-4
        dx = p * (g[rows] @ V.t() - (g[rows] * h).sum(1, keepdim=True))
        dq = dx @ K * scale
        assert float((out["dQ"][0, q, rows].double() - dq).norm() / dq.norm()) < 1e-2
    keys = torch.tensor([0, 1, 63, 64, 65, 127, 128, 5000, 18985, 19000, 20010], device="cuda")
    for k in range(Hkv):
        dk = torch.zeros(len(keys), d, dtype=torch.float64, device="cuda")
        dv = torch.zeros_like(dk)
        K, V = dev["K"][0, k].double(), dev["V"][0, k].double()
        t = torch.arange(N, device="cuda")
        for q in (2 * k, 2 * k + 1):
            Q, g = dev["Q"][0, q].double(), dev["g"][0, q].double()
            s = (keys[None] <= t[:, None]) & ((t[:, None] - keys[None] < window) | (keys[None] < sinks))
            p = torch.where(s, torch.exp(Q @ K[keys].t() * scale - out["lse"][0, q].double()[:, None]), 0.0)
            D = (g * out["h"][0, q].double()).sum(1, keepdim=True)
            dv += p.t() @ g
            dk += (p * (g @ V[keys].t() - D)).t() @ Q * scale
        for name, want in (("dK", dk), ("dV", dv)):
            got = out[name][0, k, keys].double()
            assert float(((got - want).norm(dim=1) / want.norm(dim=1)).max()) < 1e-2, name


# Logits of some hundreds whose maxima rise and fall along the keys (every raise is far above the 2^8 that the forward
# allows without one), values far from zero, and their gradients: rows alone and two 128-row tiles at a time.
LARGE = {
    "rows_alone": (1, 2, 1, 400, 64, 300, 3),
    "rows_alone_d128": (1, 2, 2, 390, 128, api.EVERYTHING, 0),
    "two_tiles": (1, 80, 8, 400, 64, 300, 3),
    "two_tiles_d128": (1, 75, 15, 385, 128, 200, 70),
}


@pytest.mark.parametrize("wave", ["rising", "rising_and_falling"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(LARGE))
def test_large_logits_and_their_gradients(name, dtype, wave):
    B, Hq, Hkv, N, d, window, sinks = LARGE[name]
    host = _inputs(B, Hq, Hkv, N, d, dtype, 31)
    u = torch.arange(N)[None, None, :, None]
    ramp = 0.1 + 12.0 * u / N if wave == "rising" else 6.0 + 6.0 * torch.sin(u / 13.0)
    host["Q"] = host["Q"].abs()
    host["K"] = (host["K"].float().abs() * ramp).to(TYPES[dtype])
    host["V"] = (host["V"].float() + 20.0).to(TYPES[dtype])
    dims = api.make_window_dims(B, Hq, Hkv, N, d, window, sinks, dtype)
    out = _run(dims, {k: v.cuda() for k, v in host.items()})
    x = {k: v.double().numpy() for k, v in host.items()}
    f = W.forward(x["Q"], x["K"], x["V"], window, sinks, 1 / math.sqrt(d), dtype)
    within("h", out["h"], f["h"], f["tol_h"])
    within("lse", out["lse"], f["lse"], f["tol_lse"])
    r, tol = W.backward(x["Q"], x["K"], x["V"], x["g"], f, window, sinks, 1 / math.sqrt(d), dtype)
    for k in r:
        within(k, out[k], r[k], tol[k])


@pytest.mark.parametrize("shape", [(1, 8, 8, 1000, 128, 128, 16), (2, 6, 2, 517, 64, 101, 7), (1, 4, 2, 700, 64, EVERYTHING, 0)])
def test_fp32_to_its_accuracy(shape):
    """The norms of the fp32 errors.  Unit-normal inputs: logits of about 1, lse of 5 to 7.  Roundings of an exponent,
    uniform, of half a step of a value up to 8 (2^-21 / 2): rms 2^-21 / sqrt(12) = 1.4e-7 each; two of them and the
    exponential (2 ulp at most: rms below 1.4e-7) give a weight 2.4e-7.  dP and D, each a sum of d terms in chunks of
    16, add two errors of d / 16 additions (rms 2^-24 / sqrt(3) sqrt(d / 16), 1e-7 at d = 128).  A gradient's sum over
    hundreds of terms adds the same once more, its terms' errors being independent: 2.4e-7, 1.4e-7 and 1e-7 in squares
    are 3e-7, and twice that is left for the correlated part (lse is one value for a row, D too).  Sums that ran in
    the tensor core, which cuts off, were 2e-6 off."""
    B, Hq, Hkv, N, d, window, sinks = shape
    host = _inputs(B, Hq, Hkv, N, d, "f32", 13)
    dims = api.make_window_dims(B, Hq, Hkv, N, d, window, sinks, "f32")
    out = _run(dims, {k: v.cuda() for k, v in host.items()})
    x = {k: v.double().numpy() for k, v in host.items()}
    f = W.forward(x["Q"], x["K"], x["V"], window, sinks, 1 / math.sqrt(d), "f32")
    r, _ = W.backward(x["Q"], x["K"], x["V"], x["g"], f, window, sinks, 1 / math.sqrt(d), "f32")
    for k, want in (("h", f["h"]), *r.items()):
        assert rel_l2(f64(out[k]), want) < 9e-7, (k, rel_l2(f64(out[k]), want))
