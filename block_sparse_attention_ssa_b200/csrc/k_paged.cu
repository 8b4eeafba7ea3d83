// The paged cache's writer, and the join of attention partials.
#include "win_common.cuh"

#include <type_traits>

namespace ssa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// Append: one pass over the new rows in 16-byte pieces.  A CTA takes ROWS packed tokens
// (all kv heads); a warp finds a token's sequence and page row, then the CTA copies.  Bound by
// memory (or by the launch, for single tokens): 4 row lengths of traffic a token and head; 11008
// tokens of 8 sequences, 8 heads, d = 128, bf16 (90 MB) take 16.7 us, 5.4 TB/s.
constexpr int AROWS = 8;
__global__ void __launch_bounds__(256) paged_append_kernel(PagedArgs a, PagedDims D, int vecs, int es) {
  __shared__ int64_t page_of[AROWS];
  __shared__ int slot_of[AROWS];
  const int row0 = blockIdx.x * AROWS, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  static_assert(AROWS == 8, "a row for each warp");
  const int row = row0 + w;
  // The first entry above the row ends its sequence, the largest one before it begins it (entries may fall: all are
  // looked at, 256 in flight, each with the length of the sequence that it ends; -1 behind the last one).
  constexpr int U = 8;
  int end = row < D.T ? -1 : 0, begin = -1;  // end: the entry's number, -1 while not found
  int last = 0, len = 0;                     // its value and length
  for (int i0 = 0; end < 0 && i0 <= D.seqs; i0 += 32 * U) {
    int q[U], n[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (i0 + 32 * k > D.seqs) break;
      const int i = i0 + 32 * k + lane;
      q[k] = i <= D.seqs ? clamp_row(a.q_start[i], D.T) : -1;
      n[k] = i <= D.seqs && i > 0 ? a.kv_len[i - 1] : 0;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (end >= 0 || i0 + 32 * k > D.seqs) break;
      const unsigned above = __ballot_sync(0xffffffffu, q[k] > row);
      const int f = above ? __ffs(above) - 1 : 32;
      if (above) {
        end = i0 + 32 * k + f;
        last = __shfl_sync(0xffffffffu, q[k], f);
        len = __shfl_sync(0xffffffffu, n[k], f);
      }
      begin = max(begin, __reduce_max_sync(0xffffffffu, lane < f ? q[k] : -1));
    }
  }
  if (lane == 0) {
    int64_t pg = -1;
    int slot = 0;
    if (end > 0) {
      const int pos = min(max(len, 0), D.max_pages * D.page) - (last - begin) + (row - begin);
      if (pos >= 0) {
        const int id = a.table[(int64_t)(end - 1) * D.max_pages + pos / D.page];
        if ((unsigned)id < (unsigned)D.num_pages) {
          pg = id;
          slot = pos % D.page;
        }
      }
    }
    page_of[w] = pg;
    slot_of[w] = slot;
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
    const long long U = batch.total<KT>();
    const long long per = share(U, ctas);
    const long long u0 = per * blockIdx.x, u1 = min(u0 + per, U);
    Cut cut{};
    if (u0 < U) {
      const Place at = batch.locate<KT>(u1 - 1);
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
