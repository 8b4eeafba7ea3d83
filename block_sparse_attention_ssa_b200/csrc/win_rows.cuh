// Rows formed anew over the pairs that the mask leaves.
//
// A tile's product multiplies hidden pairs too, with a weight of zero, and zero times a NaN or an infinity is
// NaN: one such value would spoil every row that shares a tile with a row that sees it.  So the kernels look at
// the rows that they store (one multiply-add a value), and where some are not finite, the warp that stored them forms them
// once more, here, from their visible pairs alone, in fp32 multiply-adds.  Rows that see no NaN or infinity come
// out finite; the others are what the formula says.  A pass over finite values calls nothing of this.
#pragma once

#include "win_common.cuh"

namespace ssa {

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) < __builtin_huge_valf(); }  // false for a NaN

__device__ __forceinline__ bool sees(int t, int u, int window, int sinks) { return u <= t && (t - u < window || u < sinks); }

template <typename T, int HD>
__device__ __forceinline__ float dot_row(const T* a, const T* b) {
  constexpr int V = Vec16<T>::kN;
  float s = 0.f;
#pragma unroll 2
  for (int c = 0; c < HD; c += V) {
    float x[V], y[V];
    Vec16<T>::load(a + c, x);
    Vec16<T>::load(b + c, y);
#pragma unroll
    for (int i = 0; i < V; ++i) s = fmaf(x[i], y[i], s);
  }
  return s;
}

// Whether a NaN or an infinity is among W values.
template <typename T, int W>
__device__ __forceinline__ bool spoiled(const T* a) {
  constexpr int V = Vec16<T>::kN;
  float z = 0.f;
#pragma unroll 2
  for (int c = 0; c < W; c += V) {
    float x[V];
    Vec16<T>::load(a + c, x);
#pragma unroll
    for (int i = 0; i < V; ++i) z = fmaf(x[i], 0.f, z);
  }
  return z != 0.f;  // a NaN differs from everything
}

// Where the keys of an item lie: K, V of the window form, or the pages of sequence b.
template <typename T>
struct KeyRows {
  TensorRef k, v;
  int b, kvh;
  const int32_t* table;  // null: window form
  int page, num_pages, max_pages;
  __device__ __forceinline__ const T* at(const TensorRef& x, int u) const {
    if (table == nullptr) return row_ptr<T>(x, b, kvh, u);
    const int id = table[(int64_t)b * max_pages + u / page];
    return (unsigned)id < (unsigned)num_pages ? row_ptr<T>(x, id, kvh, u % page) : nullptr;
  }
};

// The query at position t over tiles first .. last - 1 of kt.
struct RowView {
  KeyTiles kt;
  int t, first, last, window, sinks, N;  // N: keys of the window form
};

// Values that are not finite among the W columns at `out` (dtype T, or fp32 partials at `part`) of a query's row become
//   mul * sum_u 2^(c q . k_u - m) v_u
// over the keys u that it sees.  k, v, q begin at the row; columns at c0.  Warp-wide.  In the window form, rows that
// owe their state to a key that they see are left as they are without going through their keys, unless a hidden one of
// their tiles holds such values too: only tiles that the row sees in part are looked through for it.
template <typename T, int HD, int W, int KT>
__device__ void weigh_row(const KeyRows<T>& keys, const RowView& r, const T* q, T* out, float* part, int c0, float c,
                                       float m, float mul) {
  constexpr int NC = (W + 31) / 32;
  const int lane = threadIdx.x & 31;
  bool done[NC];  // finite, or NaN from a visible key
  float acc[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    acc[n] = 0.f;
    done[n] = lane + 32 * n >= W || is_finite(part != nullptr ? part[lane + 32 * n] : to_f32(out[lane + 32 * n]));
  }
  if (keys.table == nullptr) {
    bool hidden = false;
    for (int j = r.first; j < r.last; ++j) {
      const int u0 = r.kt.tile(j) * KT;
      if (u0 + KT - 1 <= r.t && (r.t - u0 < r.window || u0 + KT <= r.sinks)) continue;
      for (int u = u0 + lane; u < u0 + KT && u < r.N; u += 32)
        if (!sees(r.t, u, r.window, r.sinks)) hidden |= spoiled<T, W>(keys.at(keys.v, u) + c0);
    }
    if (!__any_sync(0xffffffffu, hidden)) return;
  }
  bool write[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) write[n] = !done[n];
  // from the newest key on: where all is NaN, the first of them ends it
  for (int j = r.last - 1; j >= r.first; --j) {
    for (int u0 = r.kt.tile(j) * KT + KT - 32, i0 = 0; i0 < KT; i0 += 32, u0 -= 32) {
      const int u = u0 + lane;
      const T* kr = sees(r.t, u, r.window, r.sinks) ? keys.at(keys.k, u) : nullptr;
      const float w = kr != nullptr ? exp2f(fmaf(dot_row<T, HD>(q, kr), c, -m)) : 0.f;
      for (unsigned rest = __ballot_sync(0xffffffffu, kr != nullptr); rest; rest &= rest - 1) {
        const int i = __ffs(rest) - 1;
        const T* vr = keys.at(keys.v, u0 + i) + c0;
        const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
        for (int n = 0; n < NC; ++n)
          if (!done[n]) acc[n] = fmaf(wi, to_f32(vr[lane + 32 * n]), acc[n]);
      }
      bool all = true;
#pragma unroll
      for (int n = 0; n < NC; ++n) all &= (done[n] |= acc[n] != acc[n]);
      if (__all_sync(0xffffffffu, all)) j = r.first, i0 = KT;
    }
  }
#pragma unroll
  for (int n = 0; n < NC; ++n)
    if (write[n]) {
      if (part != nullptr) part[lane + 32 * n] = acc[n] * mul;
      else out[lane + 32 * n] = from_f32<T>(acc[n] * mul);
    }
}

}  // namespace ssa
