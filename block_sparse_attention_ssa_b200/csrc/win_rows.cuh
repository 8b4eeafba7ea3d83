// Rows formed anew over the pairs that the mask leaves.
//
// A tile's product multiplies hidden pairs too, with a weight of zero, and zero times a NaN or an infinity is
// NaN: one such value would spoil every row that shares a tile with a row that sees it.  An fp32 operand as a pair of TF32
// values turns an infinity into a NaN besides.  So the kernels look at the rows that they store (one multiply-add a
// value), and where some are not finite, the warps that stored them form them once more, here, from their visible
// pairs alone, in fp32 multiply-adds.  Rows that see no NaN or infinity come out finite; the others are what the
// formula says.  A pass over finite values calls nothing of this.
#pragma once

#include "win_common.cuh"

#include <type_traits>

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

// f(u0, k) for each 32 keys u0 .. u0 + 31 of the view's tiles, the newest first, until it returns false; k: the lane's
// key row, null where the query does not see it.  Warp-wide.
template <typename T, int KT, typename F>
__device__ __forceinline__ void for_keys(const KeyRows<T>& keys, const RowView& r, F f) {
  for (int j = r.last - 1; j >= r.first; --j)
    for (int i = KT - 32; i >= 0; i -= 32) {
      const int u0 = r.kt.tile(j) * KT + i, u = u0 + (threadIdx.x & 31);
      if (!f(u0, sees(r.t, u, r.window, r.sinks) ? keys.at(keys.k, u) : nullptr)) return;
    }
}

// W columns of a query's row, from column c0 on, and its statistics where they lie (partials of a cut item: its maximum
// in base 2, its sum; outputs: lse, its normaliser's natural logarithm).  `out`, `part` (one of them null) begin at c0.
template <typename T>
struct RowOut {
  T* out;
  float* part;
  float *m, *l;  // of the partial
  float* lse;
};

// Forms the row anew where it is not finite.  In bf16 the statistics stand (the tensor cores hold infinities as they are)
// and only columns that are not finite are written; in fp32 all of them are.  In the bf16 window form, rows that owe their state
// to a key that they see are left without going through their keys, unless a hidden one of their tiles holds such
// values too: only tiles that the row sees in part are looked through for it.  Warp-wide.
template <typename T, int HD, int W, int KT>
__device__ __forceinline__ void mend_row(const KeyRows<T>& keys, const RowView& r, const T* q, const RowOut<T>& o, int c0, float c) {
  constexpr bool ALL = std::is_same_v<T, float>;
  constexpr int NC = (W + 31) / 32;
  const int lane = threadIdx.x & 31;
  const float l0 = o.part != nullptr ? *o.l : *o.lse;
  const bool empty = o.part != nullptr ? l0 == 0.f : l0 == kNegInf;
  bool fine = empty || is_finite(l0);
  if (!fine && !ALL) return;
  bool done[NC];  // needs nothing, or NaN from a visible key
  float acc[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    acc[n] = 0.f;
    done[n] = lane + 32 * n >= W || is_finite(o.part != nullptr ? o.part[lane + 32 * n] : to_f32(o.out[lane + 32 * n]));
    fine &= done[n];
  }
  if (__all_sync(0xffffffffu, fine)) return;
  if (!ALL && keys.table == nullptr) {
    bool hidden = false;
    for (int j = r.first; j < r.last; ++j) {
      const int u0 = r.kt.tile(j) * KT;
      if (u0 + KT - 1 <= r.t && (r.t - u0 < r.window || u0 + KT <= r.sinks)) continue;
      for (int u = u0 + lane; u < u0 + KT && u < r.N; u += 32)
        if (!sees(r.t, u, r.window, r.sinks)) hidden |= spoiled<T, W>(keys.at(keys.v, u) + c0);
    }
    if (!__any_sync(0xffffffffu, hidden)) return;
  }
  // the row's maximum and sum
  float m, mul = 1.f;
  if (o.part != nullptr && !ALL) {
    m = *o.m;
  } else {
    auto logit = [&](const T* k) { return dot_row<T, HD>(q, k) * c; };
    m = kNegInf;
    for_keys<T, KT>(keys, r, [&](int, const T* k) {
      if (k != nullptr) m = fmaxf(m, logit(k));
      return true;
    });
    float l = 0.f;
#pragma unroll
    for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
    const float ref = m == kNegInf ? 0.f : m;
    for_keys<T, KT>(keys, r, [&](int, const T* k) {
      if (k != nullptr) l += exp2f(logit(k) - ref);
      return true;
    });
#pragma unroll
    for (int i = 16; i; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
    if (o.part == nullptr) mul = l == 0.f ? 0.f : 1.0f / l;
    if (ALL && lane == 0) {
      if (o.part != nullptr) {
        *o.m = m;
        *o.l = l;
      } else {
        *o.lse = l == 0.f ? kNegInf : (m + log2f(l)) * 0.6931471805599453f;
      }
    }
    m = ref;
  }
  bool write[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    if (ALL) done[n] = lane + 32 * n >= W;
    write[n] = !done[n];
  }
  // from the newest key on: where all is NaN, the first of them ends it
  for_keys<T, KT>(keys, r, [&](int u0, const T* k) {
    const float w = k != nullptr ? exp2f(dot_row<T, HD>(q, k) * c - m) * mul : 0.f;
    for (unsigned rest = __ballot_sync(0xffffffffu, k != nullptr); rest; rest &= rest - 1) {
      const int i = __ffs(rest) - 1;
      const T* v = keys.at(keys.v, u0 + i) + c0;
      const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
      for (int n = 0; n < NC; ++n)
        if (!done[n]) acc[n] = fmaf(wi, to_f32(v[lane + 32 * n]), acc[n]);
    }
    bool all = true;
#pragma unroll
    for (int n = 0; n < NC; ++n) all &= (done[n] |= acc[n] != acc[n]);
    return !__all_sync(0xffffffffu, all);
  });
#pragma unroll
  for (int n = 0; n < NC; ++n)
    if (write[n]) {
      if (o.part != nullptr) o.part[lane + 32 * n] = acc[n];
      else o.out[lane + 32 * n] = from_f32<T>(acc[n]);
    }
}

// ---------------------------------------------------------------- gradients
// W columns of a gradient's row: which are not finite, and their sums over the visible pairs.
template <typename T, int W>
struct Columns {
  static constexpr int NC = (W + 31) / 32;
  float acc[NC];
  bool write[NC], done[NC];  // done: needs nothing, or NaN from a visible pair
  T* out;
  float* part;  // fp32 partials; one of the two is null
  // Both begin at the first column.  Returns whether the lane's columns are all finite.
  __device__ __forceinline__ bool look(T* out_, float* part_) {
    out = out_;
    part = part_;
    bool fine = true;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int c = (threadIdx.x & 31) + 32 * n;
      acc[n] = 0.f;
      done[n] = c >= W || is_finite(part != nullptr ? part[c] : to_f32(out[c]));
      write[n] = !done[n];
      fine &= done[n];
    }
    return fine;
  }
  __device__ __forceinline__ void add(float w, const T* x) {
#pragma unroll
    for (int n = 0; n < NC; ++n)
      if (!done[n]) acc[n] = fmaf(w, to_f32(x[(threadIdx.x & 31) + 32 * n]), acc[n]);
  }
  // Whether nothing is left to add in this lane.
  __device__ __forceinline__ bool settled() {
    bool all = true;
#pragma unroll
    for (int n = 0; n < NC; ++n) all &= (done[n] |= acc[n] != acc[n]);
    return all;
  }
  __device__ __forceinline__ void store(float mul) {
#pragma unroll
    for (int n = 0; n < NC; ++n)
      if (write[n]) {
        const int c = (threadIdx.x & 31) + 32 * n;
        if (part != nullptr) part[c] = acc[n];
        else out[c] = from_f32<T>(acc[n] * mul);
      }
  }
};

// Columns c0 .. c0 + W - 1 of a query's dQ, where they are not finite:
//   scale sum_u p (g . v_u + nd) k_u, p = 2^(c q . k_u + nl),
// over the keys u that it sees (nl: -lse in base 2, nd: -D).  q, g begin at the row, out at c0.  As above, the bf16 form
// goes through the row's keys only where a hidden one holds such values.  Warp-wide.
template <typename T, int HD, int W, int KT>
__device__ __forceinline__ void mend_dq_row(const KeyRows<T>& keys, const RowView& r, const T* q, const T* g, T* out, int c0, float c,
                                            float nl, float nd, float scale) {
  const int lane = threadIdx.x & 31;
  Columns<T, W> dq;
  // with a NaN in either statistic all of the row's weights are NaN
  if (__all_sync(0xffffffffu, dq.look(out, nullptr)) || nl != nl || nd != nd) return;
  if (!std::is_same_v<T, float>) {
    bool hidden = false;
    for (int j = r.first; j < r.last; ++j) {
      const int u0 = r.kt.tile(j) * KT;
      if (u0 + KT - 1 <= r.t && (r.t - u0 < r.window || u0 + KT <= r.sinks)) continue;
      for (int u = u0 + lane; u < u0 + KT && u < r.N; u += 32)
        if (!sees(r.t, u, r.window, r.sinks)) hidden |= spoiled<T, W>(keys.at(keys.k, u) + c0);
    }
    if (!__any_sync(0xffffffffu, hidden)) return;
  }
  for_keys<T, KT>(keys, r, [&](int u0, const T* k) {
    const float w = k != nullptr ? exp2f(fmaf(dot_row<T, HD>(q, k), c, nl)) * (dot_row<T, HD>(g, keys.at(keys.v, u0 + lane)) + nd) : 0.f;
    for (unsigned rest = __ballot_sync(0xffffffffu, k != nullptr); rest; rest &= rest - 1) {
      const int i = __ffs(rest) - 1;
      dq.add(__shfl_sync(0xffffffffu, w, i), keys.at(keys.k, u0 + i) + c0);
    }
    return !__all_sync(0xffffffffu, dq.settled());
  });
  dq.store(scale);
}

// Steps first .. last - 1 of key tile kt's queries (head h0 + s / nq, the nq query tiles of QT tokens from tile kt on).
struct QueryView {
  TensorRef q, g;
  const float *nl, *nd;  // -lse in base 2, -D: rows of Npad
  int b, Hq, h0, kt, nq, first, last, N, Npad, window, sinks;
};

// Columns c0 .. c0 + W - 1 of key u's dK and dV over those steps, where they are not finite:
//   scale sum_t p (g_t . v + nd_t) q_t and sum_t p g_t over the queries t that see u.
// k, v begin at the row; dk and dv look at their columns already.
template <typename T, int HD, int W, int QT>
__device__ __forceinline__ void mend_dkv_row(const QueryView& r, int u, const T* k, const T* v, Columns<T, W>& dk, Columns<T, W>& dv,
                                             int c0, float c, float scale) {
  const int lane = threadIdx.x & 31;
  // f(h, t0) for each 32 queries until it returns false
  auto for_queries = [&](auto f) {
    for (int s = r.first; s < r.last; ++s)
      for (int i = 0; i < QT; i += 32) {
        const int t0 = (r.kt + s % r.nq) * QT + i;
        if (t0 >= r.N) break;
        if (!f(r.h0 + s / r.nq, t0)) return;
      }
  };
  auto at = [&](const TensorRef& x, int h, int t) { return row_ptr<T>(x, r.b, h, t); };
  if (!std::is_same_v<T, float>) {
    bool hidden = false;
    for_queries([&](int h, int t0) {
      const int t = t0 + lane;
      if (t < r.N && !sees(t, u, r.window, r.sinks))
        hidden |= spoiled<T, W>(at(r.q, h, t) + c0) || spoiled<T, W>(at(r.g, h, t) + c0);
      return !__any_sync(0xffffffffu, hidden);
    });
    if (!__any_sync(0xffffffffu, hidden)) return;
  }
  for_queries([&](int h, int t0) {
    const int t = t0 + lane;
    const bool see = t < r.N && sees(t, u, r.window, r.sinks);
    float p = 0.f, dx = 0.f;
    if (see) {
      const int64_t o = ((int64_t)r.b * r.Hq + h) * r.Npad + t;
      p = exp2f(fmaf(dot_row<T, HD>(at(r.q, h, t), k), c, r.nl[o]));
      dx = p * (dot_row<T, HD>(at(r.g, h, t), v) + r.nd[o]);
    }
    for (unsigned rest = __ballot_sync(0xffffffffu, see); rest; rest &= rest - 1) {
      const int i = __ffs(rest) - 1;
      dk.add(__shfl_sync(0xffffffffu, dx, i), at(r.q, h, t0 + i) + c0);
      dv.add(__shfl_sync(0xffffffffu, p, i), at(r.g, h, t0 + i) + c0);
    }
    const bool a = dk.settled(), b = dv.settled();
    return !__all_sync(0xffffffffu, a && b);
  });
  dk.store(scale);
  dv.store(1.f);
}

}  // namespace ssa
