// Rows formed anew over the pairs that the mask leaves.
//
// A tile's product multiplies hidden pairs too, with a weight of zero, and zero times a NaN or an infinity is
// NaN: one such value would spoil every row that shares a tile with a row that sees it.  An fp32 operand as a pair of TF32
// values turns an infinity into a NaN besides.  So the kernels look at the rows that they store (one multiply-add a
// value), and where some are not finite, the CTA forms them once more, here, from their visible pairs alone, in fp32
// multiply-adds.  Rows that see no NaN or infinity come out finite; the others are what the formula says.  A pass over
// finite values calls nothing of this.
//
// A warp takes a row.  A group of HD / (16 bytes) lanes forms a dot product, so that a load covers whole rows (a lane
// a row took eight times the passes of each load), and 32 weights at a time go to sums of which a lane
// holds HD / 32 columns.
#pragma once

#include "win_common.cuh"

#include <type_traits>

namespace ssa {

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) < __builtin_huge_valf(); }  // false for a NaN

__device__ __forceinline__ bool sees(int t, int u, int window, int sinks) { return u <= t && (t - u < window || u < sinks); }

// A lane's 16 bytes of a row that other rows are multiplied with.
template <typename T, int HD>
struct RowPart {
  static constexpr int V = Vec16<T>::kN, LPR = HD / V, RPW = 32 / LPR;  // values of a lane, lanes of a row, rows of a load
  float x[V];
  __device__ __forceinline__ explicit RowPart(const T* row) { Vec16<T>::load(row + (threadIdx.x & 31) % LPR * V, x); }
  // Lane i: the dot product with row(i), zero where that is null.  Warp-wide.
  template <typename F>
  __device__ __forceinline__ float dots(F row) const {
    const int lane = threadIdx.x & 31;
    float mine = 0.f;
#pragma unroll 4
    for (int j = 0; j < LPR; ++j) {
      const T* r = row(j * RPW + lane / LPR);
      float y[V], s = 0.f;
      if (r != nullptr) {
        Vec16<T>::load(r + lane % LPR * V, y);
#pragma unroll
        for (int i = 0; i < V; ++i) s = fmaf(x[i], y[i], s);
      }
#pragma unroll
      for (int o = LPR / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      s = __shfl_sync(0xffffffffu, s, lane % RPW * LPR);
      if (lane / RPW == j) mine = s;
    }
    return mine;
  }
};

// A row's columns, HD / 32 to a lane: which of them are not finite, and their sums over the visible pairs.
template <typename T, int HD>
struct Columns {
  static constexpr int NC = HD / 32;
  float acc[NC];
  bool write[NC], done[NC];  // done: needs nothing, or NaN from a visible pair
  T* out;
  float* part;  // fp32 partials; one of the two is null
  __device__ __forceinline__ static int col() { return (threadIdx.x & 31) * NC; }
  __device__ __forceinline__ static void load(const float* p, float (&x)[NC]) {
#pragma unroll
    for (int n = 0; n < NC; n += 2) {
      const float2 y = *reinterpret_cast<const float2*>(p + n);
      x[n] = y.x;
      x[n + 1] = y.y;
    }
  }
  __device__ __forceinline__ static void load(const __nv_bfloat16* p, float (&x)[NC]) {
#pragma unroll
    for (int n = 0; n < NC; n += 2) {
      const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p + n));
      x[n] = y.x;
      x[n + 1] = y.y;
    }
  }
  // Both begin at the row.  Returns whether the lane's columns are finite.
  __device__ __forceinline__ bool look(T* out_, float* part_) {
    out = out_;
    part = part_;
    float x[NC];
    if (part != nullptr) load(part + col(), x);
    else load(out + col(), x);
    bool fine = true;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      acc[n] = 0.f;
      done[n] = is_finite(x[n]);
      write[n] = !done[n];
      fine &= done[n];
    }
    return fine;
  }
  // Whether the lane's open columns are NaN in a row that all of them see.
  __device__ __forceinline__ bool spoiled_by(const T* row) const {
    if (row == nullptr) return false;
    float x[NC];
    load(row + col(), x);
    bool all = true;
#pragma unroll
    for (int n = 0; n < NC; ++n) all &= done[n] || x[n] != x[n];
    return all;
  }
  // Settles the open columns that are NaN in a row that all of them see (null: all of them).
  __device__ __forceinline__ void meet(const T* row) {
    float x[NC];
    if (row != nullptr) load(row + col(), x);
#pragma unroll
    for (int n = 0; n < NC; ++n)
      if (!done[n] && (row == nullptr || x[n] != x[n])) {
        acc[n] = __int_as_float(0x7fffffff);
        done[n] = true;
      }
  }
  // acc += w_i row(i) for the set bits i; w: lane i's weight.  (Unrolled by eight, the kernels spilled.)
  template <typename F>
  __device__ __forceinline__ void add(unsigned bits, float w, F row) {
#pragma unroll 4
    for (int i = 0; i < 32; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      if (!(bits >> i & 1u)) continue;
      float x[NC];
      load(row(i) + col(), x);
#pragma unroll
      for (int n = 0; n < NC; ++n) acc[n] = fmaf(wi, x[n], acc[n]);
    }
  }
  __device__ __forceinline__ bool settled() {
    bool all = true;
#pragma unroll
    for (int n = 0; n < NC; ++n) all &= (done[n] |= acc[n] != acc[n]);
    return all;
  }
  __device__ __forceinline__ void store(float mul) const {
#pragma unroll
    for (int n = 0; n < NC; ++n)
      if (write[n]) {
        if (part != nullptr) part[col() + n] = acc[n];
        else out[col() + n] = from_f32<T>(acc[n] * mul);
      }
  }
};

// Whether a NaN or an infinity is among the values of row(0) .. row(31) (null: none).  Warp-wide.
template <typename T, int HD, typename F>
__device__ __forceinline__ bool spoiled(F row) {
  using P = RowPart<T, HD>;
  const int lane = threadIdx.x & 31;
  float z = 0.f;
#pragma unroll 4
  for (int j = 0; j < P::LPR; ++j) {
    const T* r = row(j * P::RPW + lane / P::LPR);
    if (r == nullptr) continue;
    float x[P::V];
    Vec16<T>::load(r + lane % P::LPR * P::V, x);
#pragma unroll
    for (int i = 0; i < P::V; ++i) z = fmaf(x[i], 0.f, z);
  }
  return __any_sync(0xffffffffu, z != 0.f);  // a NaN differs from everything
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

// f(u0) for each 32 keys u0 .. u0 + 31 of the view's tiles that it sees some of, the newest first, until it returns false.
template <int KT, typename F>
__device__ __forceinline__ void for_keys(const RowView& r, F f) {
  for (int j = r.last - 1; j >= r.first; --j)
    for (int i = KT - 32; i >= 0; i -= 32) {
      const int u0 = r.kt.tile(j) * KT + i;
      if (u0 > r.t || (u0 + 31 <= r.t - r.window && u0 >= r.sinks)) continue;
      if (!f(u0)) return;
    }
}

// Whether a hidden row of `x` that the view's tiles held is not finite: only tiles seen in part hold some.  Window form.
template <typename T, int HD, int KT>
__device__ __forceinline__ bool hidden_spoiled(const KeyRows<T>& keys, const TensorRef& x, const RowView& r) {
  for (int j = r.first; j < r.last; ++j) {
    const int u0 = r.kt.tile(j) * KT;
    if (u0 + KT - 1 <= r.t && (r.t - u0 < r.window || u0 + KT <= r.sinks)) continue;
    for (int u = u0; u < u0 + KT && u < r.N; u += 32)
      if (spoiled<T, HD>([&](int i) { return u + i < r.N && !sees(r.t, u + i, r.window, r.sinks) ? keys.at(x, u + i) : nullptr; }))
        return true;
  }
  return false;
}

// A query's row and its statistics where they lie: of a cut item's partial its maximum (base 2) and sum, of an output
// its lse.
template <typename T>
struct RowOut {
  T* out;
  float* part;  // one of the two is null
  float *m, *l;
  float* lse;
};

// Forms the row anew where it is not finite.  In bf16 the statistics stand (the tensor cores hold infinities as they are);
// in fp32 they are formed anew too where they are not finite.  In the bf16 window form, rows that owe their state to a key
// that they see are left without going through their keys, unless a hidden one of their tiles holds such values too.
// Warp-wide.
template <typename T, int HD, int KT>
__device__ __forceinline__ void mend_row(const KeyRows<T>& keys, const RowView& r, const T* q, const RowOut<T>& o, float c) {
  constexpr bool F32 = std::is_same_v<T, float>;
  const int lane = threadIdx.x & 31;
  float l = o.part != nullptr ? *o.l : *o.lse, m = o.part != nullptr ? *o.m : l * 1.4426950408889634f, mul = 1.f;
  const bool known = is_finite(l) || (o.part == nullptr && l == kNegInf);
  Columns<T, HD> h;
  bool fine = h.look(o.out, o.part);
  if (!known && !F32) return;
  if (__all_sync(0xffffffffu, known && fine)) return;
  // A NaN in the row's own value leaves nothing to form: inputs that are NaN throughout cost no pass over the keys.
  if (known && __all_sync(0xffffffffu, h.spoiled_by(r.t >= 0 ? keys.at(keys.v, r.t) : nullptr))) return;
  if (!F32 && keys.table == nullptr && !hidden_spoiled<T, HD, KT>(keys, keys.v, r)) return;
  const RowPart<T, HD> part(q);
  auto key = [&](int u) { return sees(r.t, u, r.window, r.sinks) ? keys.at(keys.k, u) : nullptr; };
  // the logits of keys u0 .. u0 + 31 in base 2, -infinity where the row does not see them
  auto logits = [&](int u0) {
    const float x = part.dots([&](int i) { return key(u0 + i); }) * c;
    return key(u0 + lane) != nullptr ? x : kNegInf;
  };
  if (!known) {
    m = kNegInf;
    bool nan = false;  // a visible logit is: the row's values all are, as they stand
    for_keys<KT>(r, [&](int u0) {
      const float x = logits(u0);
      m = fmaxf(m, x);
      nan = __any_sync(0xffffffffu, x != x);
      return !nan;
    });
    if (nan) return;
#pragma unroll
    for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
    const float ref = m == kNegInf ? 0.f : m;
    l = 0.f;
    for_keys<KT>(r, [&](int u0) {
      const float x = logits(u0);
      if (key(u0 + lane) != nullptr) l += exp2f(x - ref);
      return true;
    });
#pragma unroll
    for (int i = 16; i; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
    if (o.part == nullptr) mul = l == 0.f ? 0.f : 1.0f / l;
    if (lane == 0) {
      if (o.part != nullptr) {
        *o.m = m;
        *o.l = l;
      } else {
        *o.lse = l == 0.f ? kNegInf : (m + log2f(l)) * 0.6931471805599453f;
      }
    }
  }
  if (m == kNegInf) m = 0.f;
  // from the newest key on: where all is NaN, the first of them ends it
  for_keys<KT>(r, [&](int u0) {
    const float x = logits(u0);
    const unsigned bits = __ballot_sync(0xffffffffu, key(u0 + lane) != nullptr);
    h.add(bits, exp2f(x - m) * mul, [&](int i) { return keys.at(keys.v, u0 + i); });
    return !__all_sync(0xffffffffu, h.settled());
  });
  h.store(1.f);
}

// ---------------------------------------------------------------- gradients
// A query's dQ, where it is not finite:
//   scale sum_u p (g . v_u + nd) k_u, p = 2^(c q . k_u + nl),
// over the keys u that it sees (nl: -lse in base 2, nd: -D).  As above, the bf16 form goes through the row's keys
// only where a hidden one holds such values.  Warp-wide.
template <typename T, int HD, int KT>
__device__ __forceinline__ void mend_dq_row(const KeyRows<T>& keys, const RowView& r, const T* q, const T* g, T* out, float c,
                                            float nl, float nd, float scale) {
  const int lane = threadIdx.x & 31;
  Columns<T, HD> dq;
  // with a NaN in either statistic all of the row's weights are NaN
  if (__all_sync(0xffffffffu, dq.look(out, nullptr)) || nl != nl || nd != nd) return;
  if (!std::is_same_v<T, float> && !hidden_spoiled<T, HD, KT>(keys, keys.k, r)) return;
  const RowPart<T, HD> pq(q), pg(g);
  auto of = [&](const TensorRef& x, int u) { return sees(r.t, u, r.window, r.sinks) ? keys.at(x, u) : nullptr; };
  for_keys<KT>(r, [&](int u0) {
    const float x = pq.dots([&](int i) { return of(keys.k, u0 + i); });
    const float dp = pg.dots([&](int i) { return of(keys.v, u0 + i); });
    const unsigned bits = __ballot_sync(0xffffffffu, sees(r.t, u0 + lane, r.window, r.sinks));
    dq.add(bits, exp2f(fmaf(x, c, nl)) * (dp + nd), [&](int i) { return keys.at(keys.k, u0 + i); });
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

// Key u's dK and dV over those steps, where they are not finite:
//   scale sum_t p (g_t . v + nd_t) q_t and sum_t p g_t over the queries t that see u.
// Warp-wide.
template <typename T, int HD, int QT>
__device__ __forceinline__ void mend_dkv_row(const QueryView& r, int u, const T* k, const T* v, T* dk_out, T* dv_out, float* dk_part,
                                             float* dv_part, float c, float scale) {
  const int lane = threadIdx.x & 31;
  Columns<T, HD> dk, dv;
  const bool a = dk.look(dk_out, dk_part), b = dv.look(dv_out, dv_part);
  if (__all_sync(0xffffffffu, a && b)) return;
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
  auto seen = [&](int t) { return t < r.N && sees(t, u, r.window, r.sinks); };
  // A row of Q or g that is not finite shows in its query's statistics: f(h, t0, bits, nl, nd) for those of each 32 queries.
  auto for_bad = [&](bool visible, auto f) {
    for_queries([&](int h, int t0) {
      const int64_t o = ((int64_t)r.b * r.Hq + h) * r.Npad + t0 + lane;  // rows up to Npad, a multiple of 128
      const float nl = r.nl[o], nd = r.nd[o];
      const bool bad = t0 + lane < r.N && !(is_finite(nl) && is_finite(nd)) && seen(t0 + lane) == visible;
      const unsigned bits = __ballot_sync(0xffffffffu, bad);
      return bits == 0 || f(h, t0, bits, nl, nd);
    });
  };
  auto open = [](Columns<T, HD>& x) {
    const bool e = x.settled();
    return !__all_sync(0xffffffffu, e);
  };
  // A visible one with a NaN settles columns without a product.
  for_bad(true, [&](int h, int t0, unsigned bits, float nl, float nd) {
    for (; bits; bits &= bits - 1) {
      const int i = __ffs(bits) - 1;
      const float l = __shfl_sync(0xffffffffu, nl, i), d = __shfl_sync(0xffffffffu, nd, i);
      if (l != l || d != d) dk.meet(nullptr);
      dv.meet(l != l ? nullptr : at(r.g, h, t0 + i));
    }
    const bool e = open(dk), f = open(dv);
    return e || f;
  });
  bool need_k = open(dk), need_v = open(dv);
  if (!need_k && !need_v) return;
  // In bf16 the queries are gone through only where a hidden one holds such values.
  bool hidden = std::is_same_v<T, float>;
  if (!hidden)
    for_bad(false, [&](int h, int t0, unsigned bits, float, float) {
      auto of = [&](const TensorRef& x) { return [&, x, h, t0, bits](int i) { return bits >> i & 1u ? at(x, h, t0 + i) : nullptr; }; };
      hidden = spoiled<T, HD>(of(r.q)) || spoiled<T, HD>(of(r.g));
      return !hidden;
    });
  if (!hidden) return;
  const RowPart<T, HD> pk(k), pv(v);
  for_queries([&](int h, int t0) {
    const unsigned bits = __ballot_sync(0xffffffffu, seen(t0 + lane));
    if (bits == 0) return true;
    auto of = [&](const TensorRef& x) { return [&, x, h, t0](int i) { return seen(t0 + i) ? at(x, h, t0 + i) : nullptr; }; };
    const int64_t o = ((int64_t)r.b * r.Hq + h) * r.Npad + t0 + lane;
    const float p = exp2f(fmaf(pk.dots(of(r.q)), c, r.nl[o]));
    if (need_k) dk.add(bits, p * (pv.dots(of(r.g)) + r.nd[o]), [&](int i) { return at(r.q, h, t0 + i); });
    if (need_v) dv.add(bits, p, [&](int i) { return at(r.g, h, t0 + i); });
    need_k = open(dk);
    need_v = open(dv);
    return need_k || need_v;
  });
  dk.store(scale);
  dv.store(1.f);
}

}  // namespace ssa
