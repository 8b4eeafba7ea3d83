// The paged cache's writer, and the join of attention partials.
#include "win_common.cuh"

#include <type_traits>

namespace ssa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// The end entry of the sequence that holds packed row `row`, by halving: entries that do not fall.  0 for rows of no sequence.
__device__ __forceinline__ int end_by_halves(const int32_t* q_start, int seqs, int row) {
  int lo = 0, hi = seqs;  // q_start[lo] <= row < q_start[hi] once both ends hold
  if (row < q_start[0] || row >= q_start[seqs]) return 0;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (q_start[mid] <= row) lo = mid; else hi = mid;
  }
  return hi;
}

// The same where entries fall, a warp a row: the first entry above the row ends its sequence, the largest one before it
// begins it.
__device__ __forceinline__ void search_row(const int32_t* q_start, int seqs, int T, int row, int* end_of, int* begin_of) {
  const int lane = threadIdx.x & 31;
  int end = row < T ? -1 : 0, begin = 0;  // end: -1 while not found
  for (int i0 = 0; end < 0 && i0 <= seqs; i0 += 32) {
    const int q = i0 + lane <= seqs ? clamp_row(q_start[i0 + lane], T) : -1;
    const unsigned above = __ballot_sync(0xffffffffu, q > row);
    if (above) end = i0 + __ffs(above) - 1;
    begin = max(begin, __reduce_max_sync(0xffffffffu, q > row || (above && i0 + lane > end) ? -1 : q));
  }
  if (lane == 0) {
    *end_of = max(end, 0);
    *begin_of = begin;
  }
}

// Append: one pass over the new rows in 16-byte pieces.  A CTA takes ROWS packed tokens
// (all kv heads); a thread finds a token's page row once, then the CTA copies.  Bound by
// memory (or by the launch, for single tokens): 4 row lengths of traffic a token and head; 11008
// tokens of 8 sequences, 8 heads, d = 128, bf16 (90 MB) take 16.7 us, 5.4 TB/s.
// Sequences are found by halving q_start, while the CTA looks whether an entry falls; only then all are gone through
// (always so, one token of each of 4096 sequences took 35 us, this way 8.4).  The kernel wants its 30 registers: 58, with the
// placement tried before and after the search, took 33 us for 25.5 (8 sequences of 2048 new tokens).
constexpr int AROWS = 8;
__global__ void __launch_bounds__(256) paged_append_kernel(PagedArgs a, PagedDims D, int vecs, int es) {
  __shared__ int64_t page_of[AROWS];
  __shared__ int slot_of[AROWS], end_of[AROWS], begin_of[AROWS];
  const int row0 = blockIdx.x * AROWS;
  auto entry = [&](int i) { return clamp_row(a.q_start[i], D.T); };
  bool falls = false;
  if (D.seqs > 1)
    for (int i = 1 + threadIdx.x; i <= D.seqs; i += 256) falls |= entry(i) < entry(i - 1);
  int end = 0, begin = 0;  // of the thread's row: the entry that ends its sequence (0: none), the sequence's first row
  if (threadIdx.x < AROWS && row0 + threadIdx.x < D.T) {
    end = end_by_halves(a.q_start, D.seqs, row0 + threadIdx.x);
    if (end > 0) begin = entry(end - 1);
  }
  if (D.seqs > 1 && __syncthreads_or(falls)) {
    static_assert(AROWS == 8, "a row for each warp");
    const int w = threadIdx.x >> 5;
    search_row(a.q_start, D.seqs, D.T, row0 + w, &end_of[w], &begin_of[w]);
    __syncthreads();
    if (threadIdx.x < AROWS) {
      end = end_of[threadIdx.x];
      begin = begin_of[threadIdx.x];
    }
  }
  if (threadIdx.x < AROWS) {
    int64_t pg = -1;
    int slot = 0;
    if (end > 0) {
      const Seq s = load_seq(a.q_start, a.kv_len, end - 1, begin, D.T, D.max_pages * D.page);
      const int pos = s.len - s.n + (row0 + (int)threadIdx.x - s.q0);
      if (pos >= 0) {
        const int id = a.table[(int64_t)(end - 1) * D.max_pages + pos / D.page];
        if ((unsigned)id < (unsigned)D.num_pages) {
          pg = id;
          slot = pos % D.page;
        }
      }
    }
    page_of[threadIdx.x] = pg;
    slot_of[threadIdx.x] = slot;
  }
  __syncthreads();
  const int per_row = D.Hkv * vecs;
  for (int e = threadIdx.x; e < AROWS * per_row; e += 256) {
    const int r = e / per_row, h = e % per_row / vecs, c = e % vecs;
    const int64_t pg = page_of[r];
    if (pg < 0) continue;
    const int64_t row = row0 + r;
    auto piece = [&](const TensorRef& t, int64_t b, int64_t n) {
      return const_cast<uint4*>(reinterpret_cast<const uint4*>(static_cast<const char*>(t.p) + (b * t.sb + h * t.sh + n * t.sn) * es)) + c;
    };
    const uint4 k = *piece(a.nk, 0, row), v = *piece(a.nv, 0, row);
    *piece(a.k, pg, slot_of[r]) = k;
    *piece(a.v, pg, slot_of[r]) = v;
  }
}

// Join: CTA (c, y) looks whether the last item of attention CTA c is cut there and
// begins there; if so it adds that item's partials in CTA order,
//   m = max m_i, h = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i, a warp per row.
// Bound by latency (a few partials a row, from L2): 9 to 17 us alone and cold; behind the attention kernel, with
// its launch and search overlapped, one token over 65536 takes 65 us in all, 55 of them in that kernel.
template <typename T, int HD, int KT, int ROWS>
__global__ void __launch_bounds__(256) paged_join_kernel(PagedArgs a, Batch batch, int T_, int g, int ctas) {
  // Launched while the attention kernel still runs: only the partials wait for its end.  The item, by one warp:
  struct Cut {
    Seq s;
    int i0, kvh, parts, first;  // parts 0: nothing to join; first: slot of the first part
  };
  __shared__ Cut sh;
  if (threadIdx.x < 32) {
    bool falls;
    const long long U = batch.total<KT>(falls);
    const long long per = share(U, ctas);
    const long long u0 = per * blockIdx.x, u1 = min(u0 + per, U);
    Cut cut{};
    if (u0 < U) {
      const Place at = batch.locate<KT>(u1 - 1, falls);
      const long long begin = u1 - 1 - at.off;
      cut.s = load_seq(batch.q_start, batch.kv_len, at.b, at.q0, T_, batch.cap);
      cut.i0 = at.run * batch.TI;
      cut.kvh = at.kvh;
      const int units = max(1, run_tiles<KT>(cut.s, cut.i0, batch.TI, batch.window, batch.sinks).count);
      // else begun before, or complete
      if (begin >= u0 && begin + units > u1) cut.parts = 1 + (int)((begin + units - u1 + per - 1) / per);
      cut.first = 2 * blockIdx.x + (begin == u0 ? 0 : 1);
    }
    if (threadIdx.x == 0) sh = cut;
  }
  __syncthreads();
  // Every CTA waits, those without work too: what follows in the stream waits for this kernel alone.
  ahead_wait();
  const int parts = sh.parts;
  if (parts == 0) return;
  const Seq s = sh.s;
  const int i0 = sh.i0, kvh = sh.kvh, first = sh.first;
  const int nrows = min(batch.TI, s.n - i0) * g;
  const size_t psz = partial_floats(ROWS, HD);
  const float* part = static_cast<const float*>(a.ws);
  auto slot = [&](int i) { return part + psz * (i == 0 ? first : 2 * (blockIdx.x + i)); };
  const int lane = threadIdx.x & 31;
  constexpr int V = HD / 32;
  for (int r = blockIdx.y + gridDim.y * (threadIdx.x >> 5); r < nrows; r += gridDim.y * 8) {
    float m = kNegInf;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, slot(i)[ROWS * HD + r]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ref = m == kNegInf ? 0.f : m;
    float l = 0.f, o[V];
#pragma unroll
    for (int c = 0; c < V; ++c) o[c] = 0.f;
#pragma unroll 8
    for (int i = 0; i < parts; ++i) {
      const float* q = slot(i);
      const float f = exp2f(q[ROWS * HD + r] - ref);
      l = fmaf(f, q[ROWS * HD + ROWS + r], l);
#pragma unroll
      for (int c = 0; c < V; c += 2) {
        const float2 x = *reinterpret_cast<const float2*>(q + r * HD + lane * V + c);
        o[c] = fmaf(f, x.x, o[c]);
        o[c + 1] = fmaf(f, x.y, o[c + 1]);
      }
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const int h = kvh * g + r % g, row = s.q0 + i0 + r / g;
    T* dst = row_ptr_w<T>(a.h, 0, h, row) + lane * V;
#pragma unroll
    for (int c = 0; c < V; ++c) dst[c] = from_f32<T>(o[c] * inv);
    if (lane == 0) a.lse[(int64_t)h * T_ + row] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedDims& D, const PagedArgs& a, cudaStream_t st) {
  const int es = D.dtype == SSA_BF16 ? 2 : 4;
  paged_append_kernel<<<(D.T + AROWS - 1) / AROWS, 256, 0, st>>>(a, D, D.d * es / 16, es);
  count_launches(1);
  return cudaGetLastError();
}

template <int KT, int ROWS>
cudaError_t launch_paged_join(const PagedDims& D, const PagedArgs& a, int ctas, int TI, cudaStream_t st) {
  const Batch batch{a.q_start, a.kv_len, D.seqs, D.T, D.max_pages * D.page, TI, D.window, D.sinks, D.Hkv};
  // The launch and the search of the items overlap the attention kernel's last CTAs.
  using T = std::conditional_t<KT == 128, __nv_bfloat16, float>;  // units of 128 keys are the bf16 kernel's
  const dim3 grid(ctas, 4);
  return D.d == 64 ? launch_ahead(paged_join_kernel<T, 64, KT, ROWS>, grid, 256, 0, st, a, batch, D.T, D.g, ctas)
                   : launch_ahead(paged_join_kernel<T, 128, KT, ROWS>, grid, 256, 0, st, a, batch, D.T, D.g, ctas);
}
template cudaError_t launch_paged_join<128, 256>(const PagedDims&, const PagedArgs&, int, int, cudaStream_t);
template cudaError_t launch_paged_join<64, 64>(const PagedDims&, const PagedArgs&, int, int, cudaStream_t);

}  // namespace ssa
