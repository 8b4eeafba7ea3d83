"""GPU parity of ssa_paged_append and ssa_paged_attention with the 64-bit form
of oracle/window_oracle.py: ragged batches, pages of every size in either
memory order, windows, missing pages, empty rows, graphs and streams."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_ssa_b200 import api
from oracle import window_oracle as W
from tests.gpu_util import ensure_library, f64
from tests.test_gpu_window import TYPES, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


class Batch:
    """A ragged batch over scattered pages of a pool that is NaN wherever no token lies."""

    def __init__(self, new, total, Hq, Hkv, d, page, dtype, heads_first=False, seed=0, spare=3, behind=2, extra_cols=1):
        gen = torch.Generator().manual_seed(seed)
        self.new, self.total, self.Hq, self.Hkv, self.d, self.page, self.dtype = new, total, Hq, Hkv, d, page, dtype
        need = [-(-n // page) for n in total]
        self.pool = max(sum(need) + spare, 1)
        ids = torch.randperm(self.pool, generator=gen).int()
        self.cols = max(max(need), 1) + extra_cols
        self.table = torch.full((len(new), self.cols), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.q_start = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        self.kv_len = torch.tensor(total, dtype=torch.int32)
        self.T = sum(new) + behind  # rows behind the last sequence
        mk = lambda *s: torch.randn(*s, generator=gen).to(TYPES[dtype])  # noqa: E731
        self.q = mk(self.T, Hq, d)
        self.caches = []
        for _ in range(2):
            c = torch.full((self.pool, page, Hkv, d), float("nan"), dtype=TYPES[dtype])
            for b, n in enumerate(total):
                for i in range(need[b]):
                    rows = min(page, n - i * page)
                    c[self.table[b, i], :rows] = mk(rows, Hkv, d)
            self.caches.append(c)
        self.heads_first = heads_first

    def device_cache(self, c):
        if self.heads_first:
            return c.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        return c.cuda()

    def dims(self, window=None, sinks=0, scale=None):
        return api.make_paged_dims(len(self.new), self.T, self.Hq, self.Hkv, self.d, self.page, self.pool, self.cols,
                                   window, sinks, self.dtype, scale)

    def attend(self, window=None, sinks=0, table=None):
        dims = self.dims(window, sinks)
        out = {k: torch.full_like(v, 5.0) for k, v in api.alloc_paged(dims).items()}
        ws = api.alloc_paged_workspace(dims).fill_(255)
        api.ssa_paged_attention(dims, self.q.cuda(), *(self.device_cache(c) for c in self.caches), self.q_start.cuda(),
                                self.kv_len.cuda(), (self.table if table is None else table).cuda(), out["h"], out["lse"], ws)
        torch.cuda.synchronize()
        assert api.ssa_device_status() == api.SSA_OK
        return out

    def check(self, out, window=None, sinks=0, table=None):
        Kc, Vc = (np.nan_to_num(c.double().numpy()) for c in self.caches)
        r = W.paged(self.q.double().numpy(), Kc, Vc, self.q_start.numpy(), self.kv_len.numpy(),
                    (self.table if table is None else table).numpy(), self.page,
                    api.EVERYTHING if window is None else window, sinks, 1 / math.sqrt(self.d), self.dtype)
        own = r["own"]
        within("h", f64(out["h"])[own], r["h"][own], r["tol_h"][own])
        within("lse", f64(out["lse"])[:, own], r["lse"][:, own], r["tol_lse"][:, own])
        assert np.all(f64(out["h"])[~own] == 5.0) and np.all(f64(out["lse"])[:, ~own] == 5.0)


# new tokens, tokens in all, Hq, Hkv, d, page
BATCHES = {
    "one_token": ([1], [1], 1, 1, 64, 16),
    "one_long": ([1], [2500], 8, 2, 128, 64),
    "tokens": ([1] * 9, [1, 2, 16, 17, 100, 128, 129, 700, 1500], 8, 2, 128, 16),
    "some_without_new": ([0, 1, 0, 2, 0], [40, 41, 0, 300, 7], 4, 4, 64, 32),
    "chunk": ([200], [200], 4, 1, 64, 32),
    "chunks": ([70, 1, 129, 5], [500, 33, 129, 1111], 8, 2, 128, 16),
    "group_of_three": ([43, 86, 1], [100, 86, 600], 6, 2, 64, 64),
    "group_of_64": ([3, 1], [50, 400], 64, 1, 128, 128),
    "page_256": ([17, 300], [513, 700], 4, 2, 128, 256),
    "empty_rows": ([10, 5], [4, 0], 4, 2, 64, 16),
    "many_short": ([1] * 300, [1 + (7 * i) % 60 for i in range(300)], 8, 4, 64, 16),
}
VIEWS = [(None, 0), (1, 0), (50, 3), (200, 130)]


@pytest.mark.parametrize("window,sinks", VIEWS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(BATCHES))
def test_attention(name, dtype, window, sinks):
    b = Batch(*BATCHES[name], dtype, heads_first=(window == 50))
    b.check(b.attend(window, sinks), window, sinks)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_missing_pages_are_masked(dtype):
    b = Batch([30, 1, 4], [300, 200, 20], 4, 2, 64, 16, dtype)
    table = b.table.clone()
    table[0, 3], table[0, 18], table[1, 0], table[2, :] = -7, b.pool, 2**30, -1
    b.check(b.attend(None, 0, table), None, 0, table)
    b.check(b.attend(40, 20, table), 40, 20, table)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_freed_pages_are_not_used(dtype):
    """Pages behind the window are gone from the table or hold NaN: the result is the one with them in place."""
    b = Batch([20, 1], [900, 333], 8, 2, 128, 32, dtype)
    want = b.attend(100, 5)
    table = b.table.clone()
    table[0, 1:22], table[1, 1:6] = -1, -1
    got = b.attend(100, 5, table)
    for k in want:
        assert torch.equal(got[k], want[k])
    for page in torch.cat([b.table[0, 1:22], b.table[1, 1:6]]).tolist():
        for c in b.caches:
            c[page] = float("nan")
    got = b.attend(100, 5)
    for k in want:
        assert torch.equal(got[k], want[k])


def test_values_out_of_range_read_and_write_in_range():
    """q_start and kv_len past their limits are clamped: sequences that stay in range keep their results."""
    b = Batch([5, 7, 3], [100, 60, 33], 4, 2, 64, 16, "bf16", behind=0)
    want = b.attend()
    b.kv_len = torch.tensor([100, 2**31 - 1, -5], dtype=torch.int32)
    got = b.attend()
    assert torch.equal(got["h"][:5], want["h"][:5]) and bool((got["h"][12:] == 0).all())
    b.kv_len = torch.tensor([100, 60, 33], dtype=torch.int32)
    b.q_start = torch.tensor([0, 5, 2, 10**9], dtype=torch.int32)  # the second sequence has no rows, the third is cut at T
    got = b.attend()
    assert torch.equal(got["h"][:2], want["h"][:2])
    dims = b.dims()
    Kc, Vc = (b.device_cache(c) for c in b.caches)
    api.ssa_paged_append(dims, torch.ones(b.T, 2, 64, device="cuda").bfloat16(), torch.ones(b.T, 2, 64, device="cuda").bfloat16(),
                         b.q_start.cuda(), torch.tensor([-1, 2**31 - 1, 2], dtype=torch.int32).cuda(), b.table.cuda(), Kc, Vc)
    torch.cuda.synchronize()


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(BATCHES))
def test_append(name, dtype, heads_first):
    b = Batch(*BATCHES[name], dtype, heads_first=heads_first)
    if b.total[0] > 40:
        b.table[0, 2] = -1 if b.total[0] % 2 else b.pool  # a missing page: its rows go nowhere
    gen = torch.Generator().manual_seed(9)
    k, v = (torch.randn(b.T, b.Hkv, b.d, generator=gen).to(TYPES[dtype]) for _ in range(2))
    want = [c.clone() for c in b.caches]
    for i, (n, L) in enumerate(zip(b.new, b.total)):
        for j in range(n):
            pos = L - n + j
            if pos >= 0 and 0 <= int(b.table[i, pos // b.page]) < b.pool:
                for c, x in zip(want, (k, v)):
                    c[b.table[i, pos // b.page], pos % b.page] = x[int(b.q_start[i]) + j]
    got = [b.device_cache(c) for c in b.caches]
    api.ssa_paged_append(b.dims(), k.cuda(), v.cuda(), b.q_start.cuda(), b.kv_len.cuda(), b.table.cuda(), *got)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g.cpu().nan_to_num(77.0), w.nan_to_num(77.0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_serving_a_prompt_equals_the_window_forward(dtype):
    """A prompt in chunks and then token by token, appended and attended, gives the rows that the training form
    gives for the whole sequence (within the two forms' bounds)."""
    Hq, Hkv, d, page, N, window, sinks = 8, 2, 64, 16, 333, 90, 4
    gen = torch.Generator().manual_seed(1)
    Q, K, V = (torch.randn(1, h, N, d, generator=gen).to(TYPES[dtype]) for h in (Hq, Hkv, Hkv))
    x = [t.double().numpy() for t in (Q, K, V)]
    f = W.forward(*x, window, sinks, 1 / math.sqrt(d), dtype)
    pool, cols = 30, 22
    table = torch.randperm(pool, generator=gen)[:cols][None].int().cuda()
    Kc, Vc = (torch.full((pool, page, Hkv, d), float("nan"), dtype=TYPES[dtype], device="cuda") for _ in range(2))
    done = 0
    for n in [1, 130, 64, 100] + [1] * 38:
        dims = api.make_paged_dims(1, n, Hq, Hkv, d, page, pool, cols, window, sinks, dtype)
        rows = [t[0, :, done:done + n].transpose(0, 1).contiguous().cuda() for t in (Q, K, V)]
        q_start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        kv_len = torch.tensor([done + n], dtype=torch.int32, device="cuda")
        out, ws = api.alloc_paged(dims), api.alloc_paged_workspace(dims)
        api.ssa_paged_append(dims, rows[1], rows[2], q_start, kv_len, table, Kc, Vc)
        api.ssa_paged_attention(dims, rows[0], Kc, Vc, q_start, kv_len, table, out["h"], out["lse"], ws)
        within("h", f64(out["h"]).transpose(1, 0, 2), f["h"][0, :, done:done + n], f["tol_h"][0, :, done:done + n])
        within("lse", f64(out["lse"]), f["lse"][0, :, done:done + n], f["tol_lse"][0, :, done:done + n])
        done += n
    assert done == N


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_decoding_follows_the_lengths(dtype):
    """One captured step, replayed while the lengths and inputs change on the device."""
    Hq, Hkv, d, page, pool, cols, S = 8, 2, 128, 16, 80, 20, 3
    gen = torch.Generator().manual_seed(6)
    table = torch.randperm(pool, generator=gen)[:S * cols].view(S, cols).int().cuda()
    dims = api.make_paged_dims(S, S, Hq, Hkv, d, page, pool, cols, dtype=dtype)
    q, k, v = (torch.zeros(S, h, d, dtype=TYPES[dtype], device="cuda") for h in (Hq, Hkv, Hkv))
    Kc, Vc = (torch.randn(pool, page, Hkv, d, generator=gen).to(TYPES[dtype]).cuda() for _ in range(2))
    q_start = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    kv_len = torch.ones(S, dtype=torch.int32, device="cuda")
    out, ws = api.alloc_paged(dims), api.alloc_paged_workspace(dims)

    def step():
        api.ssa_paged_append(dims, k, v, q_start, kv_len, table, Kc, Vc)
        api.ssa_paged_attention(dims, q, Kc, Vc, q_start, kv_len, table, out["h"], out["lse"], ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([5, 40, 300], [6, 41, 301], [320, 1, 64]):
        kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        r = W.paged(f64(q), f64(Kc), f64(Vc), q_start.cpu().numpy(), lens, table.cpu().numpy(), page, api.EVERYTHING, 0,
                    1 / math.sqrt(d), dtype)
        within("h", out["h"], r["h"], r["tol_h"])
        within("lse", out["lse"], r["lse"], r["tol_lse"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_pages_and_fused_rows(dtype):
    """Sequences that begin with the same pages, one page twice in a sequence, and q, k, v as slices of one tensor."""
    b = Batch([40, 1, 3], [140, 97, 130], 4, 2, 64, 16, dtype)
    b.table[1, :5] = b.table[0, :5]
    b.table[2, 3] = b.table[2, 1]
    qkv = torch.full((b.T, 2 * b.Hq + 4 * b.Hkv, b.d), 7.0, dtype=TYPES[dtype])
    part = {"q": slice(0, b.Hq), "k": slice(b.Hq, b.Hq + b.Hkv), "v": slice(b.Hq + 2 * b.Hkv, b.Hq + 3 * b.Hkv)}
    host_q = b.q
    qkv[:, part["q"]] = host_q
    # the new tokens' rows, as the cache has them already (none lies in a page that is used twice)
    for name, c in zip("kv", b.caches):
        for s in range(3):
            for r in range(b.q_start[s], b.q_start[s + 1]):
                u = int(b.kv_len[s] - b.q_start[s + 1]) + r
                qkv[r, part[name]] = c[b.table[s, u // b.page], u % b.page]
    qkv = qkv.cuda()
    caches = [b.device_cache(c) for c in b.caches]
    before = [c.clone() for c in caches]
    api.ssa_paged_append(b.dims(), qkv[:, part["k"]], qkv[:, part["v"]], b.q_start.cuda(), b.kv_len.cuda(), b.table.cuda(),
                         *caches)
    for x, y in zip(before, caches):
        assert torch.equal(x.nan_to_num(9.0), y.nan_to_num(9.0))
    for window, sinks in ((None, 0), (60, 20)):
        b.q = qkv[:, part["q"]]
        out = b.attend(window, sinks)
        b.q = host_q
        b.check(out, window, sinks)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_calls_at_once(dtype):
    """Two batches on two streams, each with its own workspace, many times over."""
    batches = [Batch([1] * 5, [900, 20, 300, 77, 1200], 8, 2, 128, 16, dtype, seed=s) for s in (1, 2)]
    want = [b.attend() for b in batches]
    state = []
    for b in batches:
        dims = b.dims()
        state.append((dims, b.q.cuda(), *(b.device_cache(c) for c in b.caches), b.q_start.cuda(), b.kv_len.cuda(), b.table.cuda(),
                      {k: torch.full_like(v, 5.0) for k, v in api.alloc_paged(dims).items()}, api.alloc_paged_workspace(dims)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    for _ in range(20):
        for s, (dims, q, Kc, Vc, qs, kl, tb, out, ws) in zip(streams, state):
            api.ssa_paged_attention(dims, q, Kc, Vc, qs, kl, tb, out["h"], out["lse"], ws, stream=s)
    torch.cuda.synchronize()
    for w, st in zip(want, state):
        for k in w:
            assert torch.equal(w[k], st[7][k])


def test_cache_past_32_bit_offsets():
    """Pages whose element offsets pass 2^31."""
    page, Hkv, d, Hq = 256, 8, 128, 8
    pool = (1 << 31) // (page * Hkv * d) + 40
    Kc = torch.empty(pool, page, Hkv, d, dtype=torch.bfloat16, device="cuda")
    Vc = torch.empty_like(Kc)
    gen = torch.Generator().manual_seed(3)
    pages = [pool - 1, 3, pool - 20]
    n, L = 40, 700
    k, v, q = (torch.randn(L, h, d, generator=gen).bfloat16() for h in (Hkv, Hkv, Hq))
    table = torch.tensor([pages], dtype=torch.int32, device="cuda")
    dims = api.make_paged_dims(1, L, Hq, Hkv, d, page, pool, 3)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    api.ssa_paged_append(dims, k.cuda(), v.cuda(), ints(0, L), ints(L), table, Kc, Vc)
    dims = api.make_paged_dims(1, n, Hq, Hkv, d, page, pool, 3)
    out, ws = api.alloc_paged(dims), api.alloc_paged_workspace(dims)
    api.ssa_paged_attention(dims, q[-n:].contiguous().cuda(), Kc, Vc, ints(0, n), ints(L), table, out["h"], out["lse"], ws)
    torch.cuda.synchronize()
    small = [Kc[pages].float().cpu().numpy(), Vc[pages].float().cpu().numpy()]
    small = [np.nan_to_num(np.where(np.arange(3 * page).reshape(3, page, 1, 1) < L, c, 0.0)) for c in small]
    r = W.paged(q[-n:].double().numpy(), *small, [0, n], [L], np.array([[0, 1, 2]]), page, api.EVERYTHING, 0, 1 / math.sqrt(d), "bf16")
    within("h", out["h"], r["h"], r["tol_h"])


STARTS = {
    "as_meant": [0, 9, 11, 24, 24, 30],
    "last_falls": [0, 10, 3, 3, 3, 3],
    "falls_and_rises": [0, 5, 2, 17, 9, 30],
    "first_behind_zero": [4, 4, 1, 20, 6, 10**9],
    "negative": [-7, 12, -1, 12, 2**31 - 1, 0],
    "all_behind": [2**31 - 1, 0, 5, 7, 20, 30],
    "long": None,
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(STARTS))
def test_q_start_counts_as_its_running_maximum(name, dtype):
    """Entries that fall, pass total_q or are negative: append and attention take the same rows for each sequence, and
    no others are written, nor cache rows beside theirs."""
    Hq, Hkv, d, page, T, starts = 4, 2, 64, 16, 30, STARTS[name]
    if starts is None:  # a rise and a fall among thousands of entries
        starts = list(np.minimum(np.arange(1401) // 10, 130))
        starts[300], starts[700] = 0, 75
        T = 140
    S = len(starts) - 1
    gen = torch.Generator().manual_seed(8)
    first = np.maximum.accumulate(np.clip(np.array(starts, dtype=np.int64), 0, T))
    lens = [int(n) + 3 + 5 * (i % 7) for i, n in enumerate(np.diff(first))]
    lens[2] = 2  # rows at negative positions where it has more
    cols = -(-max(lens) // page)
    pool = S * cols + 2
    table = torch.randperm(pool, generator=gen)[:S * cols].view(S, cols).int()
    mk = lambda *s: torch.randn(*s, generator=gen).to(TYPES[dtype])  # noqa: E731
    q, k, v, caches = mk(T, Hq, d), mk(T, Hkv, d), mk(T, Hkv, d), [mk(pool, page, Hkv, d) for _ in range(2)]
    want = [c.clone() for c in caches]
    for b in range(S):
        n = int(first[b + 1] - first[b])
        for i in range(max(0, n - lens[b]), n):
            u = lens[b] - n + i
            for c, x in zip(want, (k, v)):
                c[table[b, u // page], u % page] = x[first[b] + i]
    dims = api.make_paged_dims(S, T, Hq, Hkv, d, page, pool, cols, dtype=dtype)
    ints = [torch.tensor(np.array(x), dtype=torch.int32, device="cuda") for x in (starts, lens)] + [table.cuda()]
    got = [c.cuda() for c in caches]
    api.ssa_paged_append(dims, k.cuda(), v.cuda(), *ints, *got)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), w)
    out = {n: torch.full_like(x, 5.0) for n, x in api.alloc_paged(dims).items()}
    api.ssa_paged_attention(dims, q.cuda(), *got, *ints, out["h"], out["lse"], api.alloc_paged_workspace(dims).fill_(255))
    torch.cuda.synchronize()
    assert api.ssa_device_status() == api.SSA_OK
    r = W.paged(q.double().numpy(), *(c.double().numpy() for c in want), first, lens, table.numpy(), page, api.EVERYTHING, 0,
                1 / math.sqrt(d), dtype)
    own = r["own"]
    within("h", f64(out["h"])[own], r["h"][own], r["tol_h"][own])
    within("lse", f64(out["lse"])[:, own], r["lse"][:, own], r["tol_lse"][:, own])
    assert np.all(f64(out["h"])[~own] == 5.0) and np.all(f64(out["lse"])[:, ~own] == 5.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_idle_sequences_are_passed_over(dtype):
    """Slots without new tokens before, between and behind the others: the same bits; and behind them they take no
    longer than before them (walked one at a time they took twice as long)."""
    Hq, Hkv, d, page, L, idle = 32, 8, 128, 64, 600, 4000
    cols, gen = -(-L // page), torch.Generator().manual_seed(2)
    pool = 4 * cols
    Kc, Vc = (torch.randn(pool, page, Hkv, d, generator=gen).to(TYPES[dtype]).cuda() for _ in range(2))
    q, pages = torch.randn(4, Hq, d, generator=gen).to(TYPES[dtype]).cuda(), torch.arange(pool, dtype=torch.int32).view(4, cols)

    def calls(before, between, behind):
        new = [0] * before + [1, 1] + [0] * between + [1, 1] + [0] * behind
        S = len(new)
        table = torch.full((S, cols), -1, dtype=torch.int32)
        at = [i for i, n in enumerate(new) if n]
        table[at] = pages
        ints = [torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32).cuda(),
                torch.full((S,), L, dtype=torch.int32).cuda(), table.cuda()]
        dims = api.make_paged_dims(S, 4, Hq, Hkv, d, page, pool, cols, dtype=dtype)
        out, ws = api.alloc_paged(dims), api.alloc_paged_workspace(dims)

        def call():
            api.ssa_paged_attention(dims, q, Kc, Vc, *ints, out["h"], out["lse"], ws)

        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(5):
                call()
        return out, graph, (ints, ws)  # what the graph reads lives as long

    plain = calls(0, 0, 0)[0]
    runs = [calls(idle, 0, 0), calls(0, idle, 0), calls(0, 0, idle)]
    best = [1e9] * 3
    for _ in range(5):
        for i, (_, graph, _) in enumerate(runs):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            best[i] = min(best[i], a.elapsed_time(b))
    assert api.ssa_device_status() == api.SSA_OK
    for out, _, _ in runs:
        for k in plain:
            assert torch.equal(out[k], plain[k]), k
    assert best[2] <= 1.2 * best[0] and best[1] <= 1.7 * best[0], best


# new tokens, tokens in all, Hq, Hkv, d, page: chunks of two slots, few rows, one token cut among many CTAs
LARGE = {
    "chunks": ([300, 140], [700, 140], 8, 2, 128, 64),
    "tokens": ([1, 5, 2], [600, 900, 77], 8, 2, 64, 16),
    "one_token": ([1], [9000], 8, 2, 128, 64),
    "one_long_chunk": ([70], [5000], 4, 1, 64, 32),
}


@pytest.mark.parametrize("wave", ["rising", "falling", "both"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(LARGE))
def test_large_logits(name, dtype, wave):
    """Logits of some hundreds whose maxima move along the keys: the running maximum is raised in most tiles, and the
    partials of one item differ by hundreds."""
    b = Batch(*LARGE[name], dtype)
    b.q = b.q.abs()
    for s, n in enumerate(b.total):
        u = torch.arange(n, dtype=torch.float32)
        ramp = {"rising": 0.1 + 8.0 * u / n, "falling": 8.1 - 8.0 * u / n, "both": 5.0 + 4.0 * torch.sin(u / 40.0)}[wave]
        for i in range(-(-n // b.page)):
            part = ramp[i * b.page:(i + 1) * b.page]
            rows = b.caches[0][b.table[s, i], :len(part)]
            rows.copy_((rows.float().abs() * part[:, None, None]).to(TYPES[dtype]))
    for window, sinks in ((None, 0), (400, 20)):
        b.check(b.attend(window, sinks), window, sinks)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lengths_out_of_range_are_clamped(dtype):
    """kv_len below 0 and past the table's positions: the append writes and the attention reads what the clamped
    lengths say, and every other cache row keeps its value."""
    Hq, Hkv, d, page, cols, new = 4, 2, 64, 16, 3, [5, 7, 3, 2, 60]
    S, T, gen = len(new), sum(new), torch.Generator().manual_seed(12)
    lens = [100, 2**31 - 1, -5, -2**31, cols * page + 1]
    q_start = np.concatenate([[0], np.cumsum(new)])
    pool = S * cols + 2
    table = torch.randperm(pool, generator=gen)[:S * cols].view(S, cols).int()
    mk = lambda *s: torch.randn(*s, generator=gen).to(TYPES[dtype])  # noqa: E731
    q, k, v, caches = mk(T, Hq, d), mk(T, Hkv, d), mk(T, Hkv, d), [mk(pool, page, Hkv, d) for _ in range(2)]
    L = [min(max(n, 0), cols * page) for n in lens]
    want = [c.clone() for c in caches]
    for b in range(S):
        for i in range(new[b]):
            u = L[b] - new[b] + i
            if u >= 0:
                for c, x in zip(want, (k, v)):
                    c[table[b, u // page], u % page] = x[q_start[b] + i]
    dims = api.make_paged_dims(S, T, Hq, Hkv, d, page, pool, cols, dtype=dtype)
    ints = [torch.tensor(np.array(x), dtype=torch.int32, device="cuda") for x in (q_start, lens)] + [table.cuda()]
    got = [c.cuda() for c in caches]
    api.ssa_paged_append(dims, k.cuda(), v.cuda(), *ints, *got)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), w)
    out = {n: torch.full_like(x, 5.0) for n, x in api.alloc_paged(dims).items()}
    api.ssa_paged_attention(dims, q.cuda(), *got, *ints, out["h"], out["lse"], api.alloc_paged_workspace(dims).fill_(255))
    torch.cuda.synchronize()
    assert api.ssa_device_status() == api.SSA_OK
    r = W.paged(q.double().numpy(), *(c.double().numpy() for c in want), q_start, L, table.numpy(), page, api.EVERYTHING, 0,
                1 / math.sqrt(d), dtype)
    within("h", f64(out["h"]), r["h"], r["tol_h"])
    within("lse", f64(out["lse"]), r["lse"], r["tol_lse"])
