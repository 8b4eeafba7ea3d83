// Shared by the window-attention and paged-cache kernels: validated shapes,
// which key tiles a run of queries sees, and how a ragged batch is cut into
// equal shares for the CTAs of one launch.
#pragma once

#include "ssa_internal.cuh"

namespace ssa {

// Window attention: token t sees u <= t with t - u < window or u < sinks.
struct WinDims {
  int B, Hq, Hkv, N, d, g, window, sinks;  // window and sinks at most N
  float scale;
  int dtype;
};

struct WinFwdArgs {
  TensorRef q, k, v, h;
  float* lse;
};

struct WinBwdArgs {
  TensorRef q, k, v, h, g, dq, dk, dv;
  const float* lse;
  void* ws;
};

// Serving from a paged cache.
struct PagedDims {
  int seqs, T, Hq, Hkv, d, g, page, num_pages, max_pages, window, sinks;
  float scale;
  int dtype;
};

struct PagedArgs {
  TensorRef q, k, v, h;  // q, h packed [1, Hq, T, d]; k, v caches [num_pages, Hkv, page, d]
  TensorRef nk, nv;      // append: packed [1, Hkv, T, d]
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* table;
  float* lse;
  void* ws;
};

// ---------------------------------------------------------------- kernels launched ahead
// A kernel launched by launch_ahead() may be brought up while the kernel before it in the stream still runs; every
// one of its threads calls ahead_wait() before it touches what that kernel wrote (and before it ends: what follows
// in the stream waits for the last kernel alone).  allow_ahead() in the kernel before says when.
__device__ __forceinline__ void ahead_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_ahead() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
inline cudaError_t launch_ahead(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// ---------------------------------------------------------------- key tiles of a run of queries
// The tiles of KT keys that queries at positions pmin..pmax see: the sink tiles
// 0..ns-1, then tiles lo..hi of the window (sink tiles that the window reaches
// count as window tiles).
struct KeyTiles {
  int ns, lo, count;
  __host__ __device__ int tile(int j) const { return j < ns ? j : lo + (j - ns); }
};

template <int KT>
__host__ __device__ __forceinline__ KeyTiles key_tiles(int pmin, int pmax, int window, int sinks) {
  KeyTiles k{0, 0, 0};
  if (pmax < 0) return k;
  const int first = pmin - window + 1;  // no overflow: pmin > -2^30, window < 2^31
  k.lo = first > 0 ? first / KT : 0;
  const int s = sinks < pmax + 1 ? sinks : pmax + 1;
  k.ns = (s + KT - 1) / KT;
  if (k.ns > k.lo) k.ns = k.lo;
  k.count = k.ns + pmax / KT - k.lo + 1;
  return k;
}

// Bits c < n of a word.  A row's visible columns are formed as one word and applied by selects: compared one by
// one they became a branch a column, and a partly visible tile took six times a whole one.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }

// Keys u0 .. u0 + 31 that the query at position t sees.
__device__ __forceinline__ uint32_t visible_keys(int t, int u0, int window, int sinks) {
  return bits_below(t - u0 + 1) & (~bits_below(t - window - u0 + 1) | bits_below(sinks - u0));
}
// Queries t0 .. t0 + 31 that see key u.
__device__ __forceinline__ uint32_t visible_queries(int u, int t0, int window, int sinks) {
  return ~bits_below(u - t0) & (u < sinks ? ~0u : bits_below(u + window - t0));
}
__device__ __forceinline__ float keep(uint32_t vis, int c, float x, float other) {
  float r;
  asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\tselp.f32 %0, %2, %3, p;\n\t}"
      : "=f"(r)
      : "r"(vis & (1u << c)), "f"(x), "f"(other));
  return r;
}

// ---------------------------------------------------------------- shares of a ragged batch
// Work items of one paged call: (sequence b, run of TI new tokens, kv head).
// An item is as many units as its queries see key tiles (one, to write its empty
// rows, where they see none).  Units are numbered with the kv heads innermost, then
// the runs, then the sequences; CTA c takes units [c*per, (c+1)*per), so that one
// long sequence is spread over every SM and many short ones share them evenly.
// At most the first and the last item of a CTA are cut; their rows go to partials
// that a second kernel joins in order.
struct Seq {
  int q0, n, len;  // first packed row, new tokens, tokens in the cache
};

// q_start counts as the running maximum of its values clamped to 0 .. T, so that no row has two sequences.
__device__ __forceinline__ int clamp_row(int x, int T) { return min(max(x, 0), T); }

// Sequence b; q0: the running maximum up to its own entry (the sequences before it end there).
__device__ __forceinline__ Seq load_seq(const int32_t* q_start, const int32_t* kv_len, int b, int q0, int T, int cap) {
  Seq s;
  s.q0 = q0;
  s.n = max(clamp_row(q_start[b + 1], T) - q0, 0);
  s.len = min(max(kv_len[b], 0), cap);
  return s;
}

template <int KT>
__device__ __forceinline__ KeyTiles run_tiles(const Seq& s, int i0, int TI, int window, int sinks) {
  const int p0 = s.len - s.n + i0;
  return key_tiles<KT>(p0, p0 + min(TI, s.n - i0) - 1, window, sinks);
}

template <int KT>
__device__ __forceinline__ long long seq_units(const Seq& s, int TI, int window, int sinks) {
  long long u = 0;
  for (int i0 = 0; i0 < s.n; i0 += TI) u += max(1, run_tiles<KT>(s, i0, TI, window, sinks).count);
  return u;
}

struct Place {
  int b, run, kvh;  // b = seqs: past the end
  int off;          // unit within the item
  int q0;           // first row of sequence b
};

// Warp-wide: all 32 lanes call it with the same arguments.
struct Batch {
  const int32_t* q_start;
  const int32_t* kv_len;
  int seqs, T, cap, TI, window, sinks, Hkv;

  // Lane i's sequence b0 + i (none behind the last one).  Where no entry falls each one is its own maximum; else `top` is the
  // maximum before b0 (-1 at first), then before b0 + 32.
  __device__ __forceinline__ Seq lane_seq(int b0, bool falls, int& top) const {
    const int lane = threadIdx.x & 31, b = b0 + lane;
    int a = 0, e = 0, len = 0;
    if (b < seqs) {
      a = clamp_row(q_start[b], T);
      e = clamp_row(q_start[b + 1], T);
      len = min(max(kv_len[b], 0), cap);
    }
    if (falls) {
      if (top < 0) top = __shfl_sync(0xffffffffu, a, 0);
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) e = max(e, __shfl_up_sync(0xffffffffu, e, o));
      e = max(e, top);
      a = __shfl_up_sync(0xffffffffu, e, 1);
      if (lane == 0) a = top;
      top = __shfl_sync(0xffffffffu, e, 31);
      if (b >= seqs) e = a;
    }
    return Seq{a, e - a, len};
  }

  // The first sequence from b on that has new tokens (seqs: none); q0: the rows before b.  Not warp-wide: called where a share
  // goes on in another sequence, and only there (a CTA that walked on behind its share took 50 us for a thousand idle
  // sequences: four tokens over 600 before 1000 of them 28 us, once 94; 4000: 71, once 341; around 4000: 153, once 339).
  // AT entries a step: eight in fp32 (around 4000: 222 us, one at a time 323), one in bf16, where eight saved nothing there
  // and cost registers (64 single tokens over 5048: 237 us, with eight 241).
  template <int AT>
  __device__ __forceinline__ int next_seq(int b, int q0) const {
    for (; b < seqs; b += AT) {
      int e[AT];
#pragma unroll
      for (int k = 0; k < AT; ++k) e[k] = b + k < seqs ? clamp_row(q_start[b + k + 1], T) : 0;
#pragma unroll
      for (int k = 0; k < AT; ++k)
        if (e[k] > q0) return b + k;
    }
    return seqs;
  }

  template <int KT>
  __device__ __forceinline__ long long units_of(const Seq& s) const {
    return s.n > 0 ? seq_units<KT>(s, TI, window, sinks) * Hkv : 0;
  }

  // All units; whether an entry of q_start falls below the one before it.
  template <int KT>
  __device__ long long total(bool& falls) const {
    long long u = 0;
    falls = false;
    for (;;) {
      int top = -1;
      bool down = false;
      u = 0;
      for (int b0 = 0; b0 < seqs; b0 += 32) {
        const Seq s = lane_seq(b0, falls, top);
        down |= s.n < 0;
        u += units_of<KT>(s);
      }
      if (falls || !__any_sync(0xffffffffu, down)) break;
      falls = true;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    return u;
  }

  // The item and offset of unit `at` (0 <= at < total).
  template <int KT>
  __device__ Place locate(long long at, bool falls) const {
    const int lane = threadIdx.x & 31;
    long long before = 0;
    int top = -1;
    Place p{seqs, 0, 0, 0, 0};
    for (int b0 = 0; b0 < seqs; b0 += 32) {
      const Seq own = lane_seq(b0, falls, top);
      const long long mine = units_of<KT>(own);
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + incl > at);
      if (hit) {
        const int src = __ffs(hit) - 1;
        long long rest = at - (before + __shfl_sync(0xffffffffu, incl - mine, src));
        p.b = b0 + src;
        p.q0 = __shfl_sync(0xffffffffu, own.q0, src);
        const Seq s{p.q0, __shfl_sync(0xffffffffu, own.n, src), __shfl_sync(0xffffffffu, own.len, src)};
        for (int i0 = 0; i0 < s.n; i0 += TI) {
          const int u = max(1, run_tiles<KT>(s, i0, TI, window, sinks).count);
          if (rest < (long long)u * Hkv) {
            p.run = i0 / TI;
            p.kvh = (int)(rest / u);
            p.off = (int)(rest % u);
            return p;
          }
          rest -= (long long)u * Hkv;
        }
        return p;  // not reached
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return p;
  }
};

// Units of one CTA's share.  Small calls too take as many CTAs as they have units: shares of four or more units
// meant fewer partials but longer chains (bf16, one token over 600, 8 kv heads, d = 128: 13.9 us with shares of one unit,
// 15.8 of two, 18.2 of four, 43 of sixteen; over 4000 tokens and for 16 sequences 19 to 20 with one to four).
__host__ __device__ __forceinline__ long long share(long long total, int ctas) {
  return total > 0 ? (total + ctas - 1) / ctas : 1;
}

// Partials of one cut item: `rows` accumulators of d floats (not normalised), their
// maxima (base 2, scaled) and sums.
__host__ __device__ __forceinline__ size_t partial_floats(int rows, int d) { return (size_t)rows * (d + 2); }

// ---------------------------------------------------------------- backward chunks
// Steps of key tile kt (tiles of BT tokens): g heads times the query tiles that see
// it.  A tile with more than L steps is cut into chunks whose fp32 partials a second
// kernel adds in order (sink tiles are seen by every later token).
template <int BT>
__host__ __device__ __forceinline__ int query_tiles_of(int kt, int N, int window, int sinks) {
  const int NT = (N + BT - 1) / BT;
  if (kt * BT < sinks) return NT - kt;
  const int last = (kt * BT + BT - 1 + window - 1) / BT;  // window <= N <= 2^24
  return (last < NT - 1 ? last : NT - 1) - kt + 1;
}

// Chunks to aim for, two per SM, and the steps of a chunk at least on the tensor cores (1.5 us each).  Backward in us, bf16:
// 8192 tokens, 32 heads over 8, window 1024, d = 128: 483 with 148 chunks, 484 with 296, 546 with 592; 4000 tokens, 8 heads,
// everything visible, d = 64: 110, 111, 135; 1000 tokens, 8 heads over 2, window 128: 33.0 with chunks of 2 steps
// or more, 34.5 of 8, 62 of 32, and the case before 120, 111, 95.
constexpr int kBwdChunks = 296;
constexpr int kTcMinSteps = 8;

struct ChunkPlan {
  int L, NT, chunks, partials;  // per (batch, kv head)
  int cut;                      // tiles from this one on are one chunk each
};

template <int BT>
inline ChunkPlan chunk_plan(const WinDims& D, int ctas, int min_steps) {
  ChunkPlan p{};
  p.NT = (D.N + BT - 1) / BT;
  long long steps = 0;
  for (int kt = 0; kt < p.NT; ++kt) steps += (long long)query_tiles_of<BT>(kt, D.N, D.window, D.sinks) * D.g;
  const long long all = steps * D.B * D.Hkv;
  const long long even = (all + ctas - 1) / ctas;
  // the longest shapes that the size function answers for have more steps than an int holds
  p.L = (int)(even < min_steps ? min_steps : (even < (1 << 30) ? even : 1 << 30));
  for (int kt = 0; kt < p.NT; ++kt) {
    const int n = (int)(((long long)query_tiles_of<BT>(kt, D.N, D.window, D.sinks) * D.g + p.L - 1) / p.L);
    p.chunks += n;
    if (n > 1) {
      p.partials += n;
      p.cut = kt + 1;
    }
  }
  return p;
}

struct Chunk {
  int kt, idx, n;  // chunk idx of the n of key tile kt
  int slot;        // first partial slot of the tile within its plane (n > 1)
};

// The chunk with number ci of a plane; warp-wide.  Only the first `cut` tiles are searched: behind them chunks
// and tiles go together.
template <int BT>
__device__ __forceinline__ Chunk find_chunk(int ci, int cut, int L, int g, int N, int window, int sinks) {
  const int lane = threadIdx.x & 31;
  int before = 0, slots = 0;
  Chunk r{0, 0, 1, 0};
  for (int k0 = 0; k0 < cut; k0 += 32) {
    const int kt = k0 + lane;
    const int n = kt < cut ? (int)(((long long)query_tiles_of<BT>(kt, N, window, sinks) * g + L - 1) / L) : 0;
    const int sl = n > 1 ? n : 0;
    int incl = n, incs = sl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o), z = __shfl_up_sync(0xffffffffu, incs, o);
      if (lane >= o) {
        incl += y;
        incs += z;
      }
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + incl > ci);
    if (hit) {
      const int src = __ffs(hit) - 1;
      r.kt = k0 + src;
      r.n = __shfl_sync(0xffffffffu, n, src);
      r.idx = ci - before - __shfl_sync(0xffffffffu, incl - n, src);
      r.slot = slots + __shfl_sync(0xffffffffu, incs - sl, src);
      return r;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
    slots += __shfl_sync(0xffffffffu, incs, 31);
  }
  r.kt = cut + ci - before;
  return r;
}

// ---------------------------------------------------------------- launchers
cudaError_t launch_win_fwd_f32(const WinDims& D, const WinFwdArgs& a, cudaStream_t st);

// Workspace of the backward: -lse (base 2) and -D_t in rows padded to 128 tokens, then partials.
struct WinBwdLayout {
  size_t lse2, dsum, part, bytes;
  int Npad;
};
WinBwdLayout win_bwd_layout(const WinDims& D);
// Fills lse2 (-infinity in padding rows) and dsum.
cudaError_t launch_win_bwd_pre(const WinDims& D, const WinBwdArgs& a, cudaStream_t st);
cudaError_t launch_win_bwd_f32(const WinDims& D, const WinBwdArgs& a, cudaStream_t st);
// Adds the chunks' partials of key tiles of BT tokens into dK, dV.
template <int BT>
cudaError_t launch_win_kvjoin(const WinDims& D, const WinBwdArgs& a, const ChunkPlan& p, const float* part,
                              cudaStream_t st);

cudaError_t launch_paged_append(const PagedDims& D, const PagedArgs& a, cudaStream_t st);
size_t paged_ws_bytes(const PagedDims& D);
cudaError_t launch_paged_f32(const PagedDims& D, const PagedArgs& a, cudaStream_t st);
// Joins the partials of cut items (ROWS rows of G per token of a run of TI tokens, KT keys per unit).
template <int KT, int ROWS>
cudaError_t launch_paged_join(const PagedDims& D, const PagedArgs& a, int ctas, int TI, cudaStream_t st);

// Whether rows of a bf16 tensor can be written in 32-byte pieces (a lane its row; two 16-byte pieces write half sectors
// in turn: 8192 tokens, 32 heads, d = 128, forward 176 us against 167, backward 499 against 484).
inline bool wide_rows(const TensorRef& t) {
  return reinterpret_cast<uintptr_t>(t.p) % 32 == 0 && t.sb % 16 == 0 && t.sh % 16 == 0 && t.sn % 16 == 0;
}

// TMA maps over bf16 tensors of any length with broadcast batch or head dimensions.
bool tma_map_4d(CUtensorMap* map, const void* p, int d, int64_t n1, int64_t n2, int64_t n3, int64_t s1, int64_t s2,
                int64_t s3, int b1, int b2);
bool win_tma_map(CUtensorMap* map, const TensorRef& t, int64_t B, int64_t H, int64_t N, int rows, int d, int* zero);

// bf16 on tcgen05.
cudaError_t launch_win_fwd_tc(const WinDims& D, const WinFwdArgs& a, int32_t* status, cudaStream_t st);
cudaError_t launch_win_bwd_tc(const WinDims& D, const WinBwdArgs& a, int32_t* status, cudaStream_t st);
cudaError_t launch_paged_tc(const PagedDims& D, const PagedArgs& a, int32_t* status, cudaStream_t st);
size_t paged_tc_ws_bytes(const PagedDims& D);

}  // namespace ssa
