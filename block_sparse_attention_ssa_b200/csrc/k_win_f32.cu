// Window attention with sinks and paged attention in fp32, and the preprocess and the join
// of the backward for both types.
//
// Mathematics: the online softmax over the visible keys (base 2, scale folded in) and,
// backward, p = 2^(x c - lse2), dx = p (g.v - D), dQ = scale dx K, dK = scale dx^T Q,
// dV = p^T g.  Products run on the warp-level tensor cores in TF32, each fp32 operand as the
// sum of two TF32 values (11 bits each) and each product as three: a_lo b_hi + a_hi b_lo +
// a_hi b_hi, fp32 accumulation.  What is left out, a_lo b_lo and the low part's own last
// bits, is below 2^-21 of the product: nearer than an fp32 dot product of 64 terms needs to
// be.  On the FMA pipe the same tiles were bound by shared memory (a 4 x 4 thread tile reads
// twice what the pipe can take): 178 against 142 us for a training
// step of 8 heads, 1000 tokens, d = 128, window 128.
// Measured, that step: forward 33 us, dK and dV 66 (288 chunks, two waves of CTAs), dQ 38; chunks of 120 to 301
// tokens (1051 in all) over 1200 to 3001 more, 5 sequences, 8 heads over 2, d = 64, window 1000: 89 us.  Bound by latency:
// the backward's eight warps an SM issue in 27 to 39 % of the cycles (waits for the instruction before, barriers between warps that see unequal
// parts of a tile), the tensor pipe is busy 22 to 32 %, and the fullest SM of the step above forms 1.6 times the mean's products.
// Twice the independent accumulators, or pieces twice as wide, changed nothing or spilled (134 against 134 to 144 us).
//
// Tiles: 64 queries by 64 keys, a warp 16 rows by all columns, so that a row's statistics
// need no exchange between warps and the weights go from the accumulators of one product to
// the operand of the next in registers.  Groups of four warps take a CTA's tiles in turn and
// join at the end, so that few rows fill an SM's warps too, and one group's copies
// (cp.async, zeros for hidden rows) run under another's products.
//
// Fragments of mma.m16n8k8 (g = lane / 4, t = lane % 4): A holds rows g, g + 8 and reduction
// t, t + 4; B reduction t, t + 4 and column g; C rows g, g + 8 and columns 2t, 2t + 1.  The
// order of the reduction is free: t and t + 4 stand for elements 2t and 2t + 1 of each eight,
// so an accumulator is the next product's A as it is, and A and B of the logits are 8-byte
// loads.
#include "win_rows.cuh"

#include "mma_sync.cuh"

namespace ssa {
namespace {

constexpr int BT = 64;
constexpr int GROUP = 128;  // threads on one 64 x 64 tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kPagedCtas = 148;  // CTAs of one paged call, one per SM
// Steps of a backward chunk at least: a 64 x 64 step takes microseconds of a CTA, a partial's round trip less (1000
// tokens, 8 heads, window 128, d = 128: 102 us with 2, 110 with 1, 154 with 8).
constexpr int kMinSteps = 2;

// Row pitches in shared memory, by the fragments' 32 banks: rows read as 8-byte pairs of a row (logits) want a
// pitch of 8 mod 32, rows read down a column (weighted sums) 4 mod 32.  A tile read both ways takes the latter.
template <int HD>
struct Pitch {
  static constexpr int along = HD + 8, down = HD + 4;
};

struct F32Params {
  TensorRef q, k, v, h;
  float* lse;
  int Hq, g, N, window, sinks, NT;
  float c;
  // paged
  const int32_t* table;
  Batch batch;
  int page, num_pages, max_pages, T;
  float* part;
};

// ---------------------------------------------------------------- TF32 in pairs
struct Pair {
  uint32_t hi, lo;
};
// x = hi + lo: hi rounded to 11 bits, lo the exact rest (the tensor core reads its upper 11 bits).
__device__ __forceinline__ Pair split(float x) {
  Pair p;
  p.hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  p.lo = __float_as_uint(x - __uint_as_float(p.hi));
  return p;
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c[n] += a b[n] over 16 terms to fp32 accuracy, the small terms first; the accumulators in turn, so that no
// product waits for the one before.  The tensor core cuts off what it adds to its accumulator, so sixteen terms are
// summed there and added here, rounded: running sums in the tensor core left a training step's gradients 2e-6 off
// (norms), this leaves 3e-7 to 6e-7.
template <int N>
__device__ __forceinline__ void mma_pairs(float (*c)[4], const Pair (&a)[2][4], const Pair (&b)[2][N][2]) {
  float s[N][4];
#pragma unroll
  for (int n = 0; n < N; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int n = 0; n < N; ++n) mma_tf32(s[n], a[k][0].lo, a[k][1].lo, a[k][2].lo, a[k][3].lo, b[k][n][0].hi, b[k][n][1].hi);
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int n = 0; n < N; ++n) mma_tf32(s[n], a[k][0].hi, a[k][1].hi, a[k][2].hi, a[k][3].hi, b[k][n][0].lo, b[k][n][1].lo);
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int n = 0; n < N; ++n) mma_tf32(s[n], a[k][0].hi, a[k][1].hi, a[k][2].hi, a[k][3].hi, b[k][n][0].hi, b[k][n][1].hi);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[n][i] += s[n][i];
}

// c[n] = (16 rows of A) . (rows 8 n .. 8 n + 7 of B) over HD, n < 4; A: row g of the warp's sixteen at A + g PA.
template <int HD, int PA, int PB>
__device__ __forceinline__ void logits(float (*c)[4], const float* A, const float* B, int g, int t) {
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[n][i] = 0.f;
#pragma unroll 1
  for (int k0 = 0; k0 < HD; k0 += 16) {
    Pair a[2][4], b[2][4][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 x = *reinterpret_cast<const float2*>(A + g * PA + k0 + 8 * k + 2 * t);
      const float2 y = *reinterpret_cast<const float2*>(A + (g + 8) * PA + k0 + 8 * k + 2 * t);
      a[k][0] = split(x.x);
      a[k][1] = split(y.x);
      a[k][2] = split(x.y);
      a[k][3] = split(y.y);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float2 z = *reinterpret_cast<const float2*>(B + (8 * n + g) * PB + k0 + 8 * k + 2 * t);
        b[k][n][0] = split(z.x);
        b[k][n][1] = split(z.y);
      }
    }
    mma_pairs<4>(c, a, b);
  }
}

// acc[n] += W X for the weights W (16 x 32, accumulator layout) and 32 rows of X, columns 8 n ...
template <int HD, int PX>
__device__ __forceinline__ void weighted(float (&acc)[HD / 8][4], const float (*w)[4], const float* X, int g, int t) {
#pragma unroll
  for (int k0 = 0; k0 < 4; k0 += 2) {
    Pair a[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      a[k][0] = split(w[k0 + k][0]);
      a[k][1] = split(w[k0 + k][2]);
      a[k][2] = split(w[k0 + k][1]);
      a[k][3] = split(w[k0 + k][3]);
    }
    const float* r0 = X + (8 * k0 + 2 * t) * PX + g;
#pragma unroll
    for (int n0 = 0; n0 < HD / 8; n0 += 2) {
      Pair b[2][2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          b[k][n][0] = split(r0[8 * k * PX + 8 * (n0 + n)]);
          b[k][n][1] = split(r0[(8 * k + 1) * PX + 8 * (n0 + n)]);
        }
      mma_pairs<2>(acc + n0, a, b);
    }
  }
}

// Whether a query at positions t0 .. t1 sees a key of u0 .. u0 + 31: warps leave out the others.
__device__ __forceinline__ bool any_sees(int t0, int t1, int u0, int window, int sinks) {
  return u0 <= t1 && (u0 + 31 > t0 - window || u0 < sinks);
}

// ---------------------------------------------------------------- shared memory
// 64 rows of HD values by the `n` threads tid = 0 ..; a null row gives zeros (and a copy of no bytes from `any`).
// Asynchronous: copies_done() below.
template <int HD, int P, typename F>
__device__ __forceinline__ void copy_rows(float* dst, const void* any, int tid, int n, F row) {
  constexpr int PER = HD / 4;
  for (int e = tid; e < BT * PER; e += n) {
    const float* r = row(e / PER);
    warp_mma::cp_async16(dst + (e / PER) * P + (e % PER) * 4, r != nullptr ? r + (e % PER) * 4 : any, r != nullptr ? 16 : 0);
  }
  warp_mma::cp_async_commit();
}
__device__ __forceinline__ void copies_done() { warp_mma::cp_async_wait<0>(); }
__device__ __forceinline__ void group_sync(int grp) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(GROUP) : "memory");
}

// ================================================================ forward
template <int HD>
struct Fwd {
  static constexpr int GROUPS = HD == 128 ? 3 : 4;  // registers: 168 and 128 a thread
  static constexpr int THREADS = GROUPS * GROUP;
  static constexpr int TILEF = BT * Pitch<HD>::along;
  static constexpr size_t SMEM = (size_t)(1 + GROUPS) * TILEF * 4;  // Q, then each group's K or V
};

// One item of the paged form (a share of it), or the CTA's tile of the window form.
struct F32Item {
  int b, head0, q0row, kvh, nrows, p0, per_tok, units, take, len;
  KeyTiles kt;
};

template <bool PAGED>
__device__ __forceinline__ F32Item item_of(const F32Params& p, const Place& at, int left) {
  F32Item I;
  if (PAGED) {
    const Seq s = load_seq(p.batch.q_start, p.batch.kv_len, at.b, at.q0, p.T, p.batch.cap);
    const int i0 = at.run * p.batch.TI;
    I.b = at.b;
    I.kvh = at.kvh;
    I.head0 = at.kvh * p.g;
    I.per_tok = p.g;
    I.nrows = min(p.batch.TI, s.n - i0) * p.g;
    I.q0row = s.q0 + i0;
    I.p0 = s.len - s.n + i0;
    I.len = s.len;
    I.kt = run_tiles<BT>(s, i0, p.batch.TI, p.window, p.sinks);
    I.units = max(1, I.kt.count);
    I.take = min(left, I.units - at.off);
  } else {
    const int planes = (int)(gridDim.x / p.NT);
    const int plane = (int)blockIdx.x % planes, qt = p.NT - 1 - (int)blockIdx.x / planes;
    I.b = plane / p.Hq;
    I.head0 = plane % p.Hq;
    I.kvh = I.head0 / p.g;
    I.per_tok = 1;
    I.q0row = I.p0 = qt * BT;
    I.nrows = min(BT, p.N - I.p0);
    I.len = p.N;
    I.kt = key_tiles<BT>(I.p0, I.p0 + I.nrows - 1, p.window, p.sinks);
    I.units = I.take = I.kt.count;
  }
  return I;
}

// The place behind `take` units of an item: whether the share holds more.
__device__ __forceinline__ bool next_item(const F32Params& p, Place& at, int& left, int take) {
  left -= take;
  if (left <= 0) return false;
  at.off = 0;
  if (++at.kvh == p.batch.Hkv) {
    at.kvh = 0;
    const Seq s = load_seq(p.batch.q_start, p.batch.kv_len, at.b, at.q0, p.T, p.batch.cap);
    if (++at.run * p.batch.TI >= s.n) {
      at.run = 0;
      at.q0 += s.n;
      at.b = p.batch.next_seq<8>(at.b + 1, at.q0);
    }
  }
  return at.b < p.batch.seqs;
}

// The CTA's rows once more (win_rows.cuh), those that are not finite; a warp takes every n-th row.
template <int HD, bool PAGED>
__device__ __forceinline__ void form_again(const F32Params& p, Place at, int left) {
  for (int seg = 0;; ++seg) {
    const F32Item I = item_of<PAGED>(p, at, left);
    const KeyRows<float> keys{p.k, p.v, I.b, I.kvh, PAGED ? p.table : nullptr, p.page, p.num_pages, p.max_pages};
    for (int r = threadIdx.x >> 5; r < I.nrows; r += blockDim.x >> 5) {
      const int tok = PAGED ? r / I.per_tok : r, head = PAGED ? I.head0 + r % I.per_tok : I.head0, row = I.q0row + tok;
      const int first = PAGED ? at.off : 0;
      const RowView view{I.kt, I.p0 + tok, first, min(first + I.take, I.kt.count), p.window, p.sinks, p.N};
      RowOut<float> o{};
      if (PAGED && I.take < I.units) {
        float* base = p.part + (size_t)(2 * blockIdx.x + (seg ? 1 : 0)) * partial_floats(BT, HD);
        o.part = base + r * HD;
        o.m = base + BT * HD + r;
        o.l = o.m + BT;
      } else {
        o.out = row_ptr_w<float>(p.h, PAGED ? 0 : I.b, head, row);
        o.lse = p.lse + (PAGED ? (int64_t)head * p.T + row : ((int64_t)I.b * p.Hq + I.head0) * p.N + row);
      }
      mend_row<float, HD, BT>(keys, view, row_ptr<float>(p.q, PAGED ? 0 : I.b, head, row), o, p.c);
    }
    if (!PAGED || !next_item(p, at, left, I.take)) return;
  }
}

template <int HD, bool PAGED>
__global__ void __launch_bounds__(Fwd<HD>::THREADS, 1) win_fwd_f32_kernel(F32Params p) {
  using C = Fwd<HD>;
  constexpr int PA = Pitch<HD>::along, PD = Pitch<HD>::down;
  extern __shared__ float sm[];
  float* sQ = sm;
  const int grp = threadIdx.x / GROUP, tid = threadIdx.x % GROUP, warp = tid >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  float* sX = sQ + (1 + grp) * C::TILEF;  // K, then V, at the end the group's accumulators
  __shared__ Place sh_place;
  __shared__ int sh_left;
  __shared__ float sh_m[C::GROUPS][BT], sh_l[C::GROUPS][BT];

  Place at{0, 0, 0, 0, 0};
  int left = 1;
  bool again = false;  // rows that are not finite were stored (a store to shared memory there held up the next row: 97 us for 92)
  if (PAGED) {
    if (threadIdx.x < 32) {
      bool falls;
      const long long U = p.batch.total<BT>(falls);
      const long long per = share(U, (int)gridDim.x);
      const long long u0 = per * blockIdx.x;
      const long long n = u0 < U ? min(per, U - u0) : 0;
      if (n > 0) at = p.batch.locate<BT>(u0, falls);
      if (threadIdx.x == 0) {
        sh_place = at;
        sh_left = (int)n;
      }
    }
    __syncthreads();
    allow_ahead();  // the join
    at = sh_place;
    left = sh_left;
  }

  for (int seg = 0; left > 0; ++seg) {
    // ---- the item
    const F32Item I = item_of<PAGED>(p, at, left);
    const int b = I.b, head0 = I.head0, q0row = I.q0row, kvh = I.kvh, nrows = I.nrows, p0 = I.p0, per_tok = I.per_tok;
    const int take = I.take, units = I.units, len = I.len;
    const KeyTiles kt = I.kt;
    const bool cut = PAGED && take < units;
    auto tok_of = [&](int r) { return PAGED ? r / per_tok : r; };
    auto head_of = [&](int r) { return PAGED ? head0 + r % per_tok : head0; };
    copy_rows<HD, PA>(sQ, p.q.p, threadIdx.x, C::THREADS, [&](int r) -> const float* {
      return r < nrows ? row_ptr<float>(p.q, PAGED ? 0 : b, head_of(r), q0row + tok_of(r)) : nullptr;
    });

    // rows r and r + 8 of the tile
    const int r0 = 16 * warp + g;
    float acc[HD / 8][4], m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};
    int pos[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) pos[i] = r0 + 8 * i < nrows ? p0 + tok_of(r0 + 8 * i) : -1;
#pragma unroll
    for (int n = 0; n < HD / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    const int pmax = p0 + tok_of(nrows - 1), lo_min = p0 - p.window + 1;
    const int w0 = p0 + tok_of(16 * warp), w1 = p0 + tok_of(min(16 * warp + 15, nrows - 1));  // the warp's positions

    const int end = min(at.off + take, kt.count);
    copies_done();
    __syncthreads();  // Q is there
    for (int j = at.off + grp; j < end; j += C::GROUPS) {
      const int u0 = kt.tile(j) * BT;
      // A key that no row of the item sees is not read (its memory may hold anything).
      auto keys = [&](const TensorRef& x) {
        return [&, x](int r) -> const float* {
          const int u = u0 + r;
          if (u > pmax || u >= len || (u < lo_min && u >= p.sinks)) return nullptr;
          if (!PAGED) return row_ptr<float>(x, b, kvh, u);
          const int pg = p.table[(int64_t)b * p.max_pages + u / p.page];
          return (unsigned)pg < (unsigned)p.num_pages ? row_ptr<float>(x, pg, kvh, u % p.page) : nullptr;
        };
      };
      copy_rows<HD, PA>(sX, p.q.p, tid, GROUP, keys(p.k));
      uint32_t gone[2] = {0u, 0u};  // keys whose page is missing
      if (PAGED)
        for (int c = 0; c < BT; c += 16) {  // a page holds 16 tokens at least
          const int u = u0 + c;
          if (u < len && (unsigned)p.table[(int64_t)b * p.max_pages + u / p.page] >= (unsigned)p.num_pages)
            gone[c >> 5] |= 0xffffu << (c & 16);
        }
      copies_done();
      group_sync(grp);
      float x[8][4];
      bool some[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        some[c] = any_sees(w0, w1, u0 + 32 * c, p.window, p.sinks);
        if (some[c]) {
          logits<HD, PA, PA>(x + 4 * c, sQ + 16 * warp * PA, sX + 32 * c * PA, g, t);
        } else {
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * c + n][e] = 0.f;  // masked below
        }
      }
      group_sync(grp);  // K is read
      copy_rows<HD, PD>(sX, p.q.p, tid, GROUP, keys(p.v));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t v0 = visible_keys(pos[i], u0, p.window, p.sinks) & ~gone[0];
        const uint32_t v1 = visible_keys(pos[i], u0 + 32, p.window, p.sinks) & ~gone[1];
        float mx = kNegInf;
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t vis = (n < 4 ? v0 : v1) >> (2 * t);
            x[n][2 * i + e] = keep(vis, 8 * (n & 3) + e, x[n][2 * i + e] * p.c, kNegInf);
            mx = fmaxf(mx, x[n][2 * i + e]);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[i], mx), ref = mn == kNegInf ? 0.f : mn, f = exp2f(m[i] - ref);
        m[i] = mn;
        l[i] *= f;
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[n][2 * i + e] = exp2f(x[n][2 * i + e] - ref);
            l[i] += x[n][2 * i + e];
          }
#pragma unroll
        for (int n = 0; n < HD / 8; ++n) {
          acc[n][2 * i] *= f;
          acc[n][2 * i + 1] *= f;
        }
      }
      copies_done();
      group_sync(grp);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (some[c]) weighted<HD, PD>(acc, x + 4 * c, sX + 32 * c * PD, g, t);
      group_sync(grp);  // V is read
    }

    // ---- the groups' softmaxes, joined by the first one
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      const int r = r0 + 8 * i;
      if (grp > 0) {
        if (t == 0) {
          sh_m[grp][r] = m[i];
          sh_l[grp][r] = l[i];
        }
#pragma unroll
        for (int n = 0; n < HD / 8; ++n)
          *reinterpret_cast<float2*>(sX + r * PA + 8 * n + 2 * t) = make_float2(acc[n][2 * i], acc[n][2 * i + 1]);
      }
    }
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + 8 * i;
#pragma unroll 1
        for (int o = 1; o < C::GROUPS; ++o) {
          const float m1 = sh_m[o][r], mn = fmaxf(m[i], m1), ref = mn == kNegInf ? 0.f : mn;
          const float f0 = exp2f(m[i] - ref), f1 = exp2f(m1 - ref);
          l[i] = l[i] * f0 + sh_l[o][r] * f1;
          m[i] = mn;
          const float* other = sQ + (1 + o) * C::TILEF + r * PA + 2 * t;
#pragma unroll
          for (int n = 0; n < HD / 8; ++n) {
            const float2 y = *reinterpret_cast<const float2*>(other + 8 * n);
            acc[n][2 * i] = acc[n][2 * i] * f0 + y.x * f1;
            acc[n][2 * i + 1] = acc[n][2 * i + 1] * f0 + y.y * f1;
          }
        }
        // ---- epilogue
        if (r >= nrows) continue;
        float* dst;
        float mul = 1.f;
        if (cut) {
          float* base = p.part + (size_t)(2 * blockIdx.x + (seg ? 1 : 0)) * partial_floats(BT, HD);
          dst = base + r * HD;
          if (t == 0) {
            base[BT * HD + r] = m[i];
            base[BT * HD + BT + r] = l[i];
          }
        } else {
          mul = l[i] == 0.f ? 0.f : 1.0f / l[i];
          dst = row_ptr_w<float>(p.h, PAGED ? 0 : b, head_of(r), q0row + tok_of(r));
          if (t == 0) {
            const int64_t o = PAGED ? (int64_t)head_of(r) * p.T + q0row + tok_of(r)
                                    : ((int64_t)b * p.Hq + head0) * p.N + q0row + r;
            p.lse[o] = l[i] == 0.f ? kNegInf : (m[i] + log2f(l[i])) * kLn2;
          }
        }
        float z = l[i] * 0.f;
#pragma unroll
        for (int n = 0; n < HD / 8; ++n) {
          const float2 y = make_float2(acc[n][2 * i] * mul, acc[n][2 * i + 1] * mul);
          *reinterpret_cast<float2*>(dst + 8 * n + 2 * t) = y;
          z = fmaf(y.x, 0.f, fmaf(y.y, 0.f, z));
        }
        again |= z != 0.f;
      }
    }
    if (!PAGED) break;
    // ---- the next item
    if (!next_item(p, at, left, take)) break;
    __syncthreads();  // shared memory is read to the end
  }
  if (__syncthreads_or(again)) form_again<HD, PAGED>(p, PAGED ? sh_place : Place{0, 0, 0, 0, 0}, PAGED ? sh_left : 1);
}

// ================================================================ backward
// -D_t = -(g_t . h_t) and -lse in base 2, rows padded to 128 tokens.  Bound by reading h and g: a row is LPR
// lanes of 16 bytes, and a warp has four rows' loads of each in flight per lane group.  32 heads of 16384 tokens,
// d = 128, bf16 (270 MB): 50 us, 5.5 TB/s.
template <typename T, int HD>
__global__ void __launch_bounds__(256) win_bwd_pre_kernel(TensorRef h, TensorRef g, const float* lse, float* lse2,
                                                          float* dsum, int Hq, int N, int Npad) {
  constexpr int V = Vec16<T>::kN, LPR = HD / V, RPW = 32 / LPR, U = 4;
  const int lane = threadIdx.x & 31, c = lane % LPR * V;
  const int bh = blockIdx.y, b = bh / Hq, hd = bh % Hq;
  const int t0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * (RPW * U) + lane / LPR;
  allow_ahead();
  uint4 x[U], y[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int t = t0 + i * RPW;
    x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
    if (t < N) {
      x[i] = *reinterpret_cast<const uint4*>(row_ptr<T>(h, b, hd, t) + c);
      y[i] = *reinterpret_cast<const uint4*>(row_ptr<T>(g, b, hd, t) + c);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int t = t0 + i * RPW;
    float u[V], v[V], s = 0.f;
    Vec16<T>::load(reinterpret_cast<const T*>(&x[i]), u);
    Vec16<T>::load(reinterpret_cast<const T*>(&y[i]), v);
#pragma unroll
    for (int e = 0; e < V; ++e) s = fmaf(u[e], v[e], s);
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane % LPR == 0 && t < Npad) {
      float ls = kNegInf;  // 2^(x - inf) = 0 in the padding and in rows without weight
      if (t < N) {
        const float l = lse[(int64_t)bh * N + t] * kLog2e;
        if (l != kNegInf) ls = -l;
      }
      lse2[(int64_t)bh * Npad + t] = ls;
      dsum[(int64_t)bh * Npad + t] = -s;
    }
  }
}

struct F32Bwd {
  TensorRef q, k, v, g, dq, dk, dv;
  const float* lse2;
  const float* dsum;
  float* part;
  int Hq, Hkv, grp, N, Npad, window, sinks, NT, L, partials, cut;
  float c, scale;
};

// Two groups of four warps, up to 255 registers a thread, for the accumulators of a warp's sixteen rows (128 in dkv at
// d = 128, where 312 bytes are spilled all the same; dq there 36); logits and dP are formed 32 columns at a time.
constexpr int BWD_THREADS = 2 * GROUP;

// dq: Q, g, then each group's K, V.  dkv: K, V, then each group's Q, g.
template <int HD>
constexpr size_t bwd_smem() {
  return (size_t)(2 * BT * Pitch<HD>::along + 2 * BT * (Pitch<HD>::down + Pitch<HD>::along)) * 4;
}

// The second group's accumulators are added to the first's through shared memory (the group's own tiles).
template <int HD>
__device__ __forceinline__ void add_groups(float (&acc)[HD / 8][4], float* buf, int grp, int r0, int t) {
  constexpr int P = Pitch<HD>::down;
  __syncthreads();
#pragma unroll
  for (int n = 0; n < HD / 8; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float2* q = reinterpret_cast<float2*>(buf + (r0 + 8 * i) * P + 8 * n + 2 * t);
      if (grp == 1) *q = make_float2(acc[n][2 * i], acc[n][2 * i + 1]);
    }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < HD / 8; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 y = *reinterpret_cast<const float2*>(buf + (r0 + 8 * i) * P + 8 * n + 2 * t);
      if (grp == 0) {
        acc[n][2 * i] += y.x;
        acc[n][2 * i + 1] += y.y;
      }
    }
}

// Returns whether a stored value is not finite.
template <int HD>
__device__ __forceinline__ bool store_rows(float* row, const float (&acc)[HD / 8][4], int i, int t, float mul) {
  float z = 0.f;
#pragma unroll
  for (int n = 0; n < HD / 8; ++n) {
    const float2 y = make_float2(acc[n][2 * i] * mul, acc[n][2 * i + 1] * mul);
    *reinterpret_cast<float2*>(row + 8 * n + 2 * t) = y;
    z = fmaf(y.x, 0.f, fmaf(y.y, 0.f, z));
  }
  return z != 0.f;
}

template <int HD>
__global__ void __launch_bounds__(BWD_THREADS, 1) win_bwd_dq_f32_kernel(F32Bwd p) {
  constexpr int PA = Pitch<HD>::along, PD = Pitch<HD>::down;
  extern __shared__ float sm[];
  const int grp = threadIdx.x / GROUP, tid = threadIdx.x % GROUP, warp = tid >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3, r0 = 16 * warp + g;
  float* sQ = sm;
  float* sG = sQ + BT * PA;
  float* sK = sG + BT * PA + grp * BT * (PD + PA);  // read along (logits) and down (dQ)
  float* sV = sK + BT * PD;
  const int planes = (int)(gridDim.x / p.NT);
  const int plane = (int)blockIdx.x % planes, qt = p.NT - 1 - (int)blockIdx.x / planes;
  const int b = plane / p.Hq, h = plane % p.Hq, kvh = h / p.grp;
  const int q0 = qt * BT, nrows = min(BT, p.N - q0);
  const KeyTiles kt = key_tiles<BT>(q0, q0 + nrows - 1, p.window, p.sinks);
  auto query = [&](const TensorRef& x) {
    return [&, x](int r) -> const float* { return r < nrows ? row_ptr<float>(x, b, h, q0 + r) : nullptr; };
  };
  copy_rows<HD, PA>(sQ, p.q.p, threadIdx.x, BWD_THREADS, query(p.q));
  copy_rows<HD, PA>(sG, p.q.p, threadIdx.x, BWD_THREADS, query(p.g));
  ahead_wait();
  float nl[2], nd[2], acc[HD / 8][4];  // -lse2, -D
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t o = ((int64_t)b * p.Hq + h) * p.Npad + q0 + r0 + 8 * i;
    nl[i] = p.lse2[o];
    nd[i] = p.dsum[o];
  }
#pragma unroll
  for (int n = 0; n < HD / 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  copies_done();
  __syncthreads();
  for (int j = grp; j < kt.count; j += 2) {
    const int u0 = kt.tile(j) * BT;
    // keys that no query of the tile sees are not read
    auto key = [&](const TensorRef& x) {
      return [&, x](int r) -> const float* {
        const int u = u0 + r;
        return u < q0 + nrows && (u > q0 - p.window || u < p.sinks) ? row_ptr<float>(x, b, kvh, u) : nullptr;
      };
    };
    copy_rows<HD, PD>(sK, p.q.p, tid, GROUP, key(p.k));
    copy_rows<HD, PA>(sV, p.q.p, tid, GROUP, key(p.v));
    copies_done();
    group_sync(grp);
#pragma unroll 1
    for (int c0 = 0; c0 < BT; c0 += 32) {
      float x[4][4], y[4][4];
      if (!any_sees(q0 + 16 * warp, q0 + 16 * warp + 15, u0 + c0, p.window, p.sinks)) continue;
      logits<HD, PA, PD>(x, sQ + 16 * warp * PA, sK + c0 * PD, g, t);
      logits<HD, PA, PA>(y, sG + 16 * warp * PA, sV + c0 * PA, g, t);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t vis = visible_keys(q0 + r0 + 8 * i, u0 + c0, p.window, p.sinks) >> (2 * t);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = 2 * i + e;
            x[n][k] = keep(vis, 8 * n + e, exp2f(fmaf(x[n][k], p.c, nl[i])) * (y[n][k] + nd[i]), 0.f);
          }
      }
      weighted<HD, PD>(acc, x, sK + c0 * PD, g, t);
    }
    group_sync(grp);  // K and V are read
  }
  add_groups<HD>(acc, sG + BT * PA, grp, r0, t);
  bool again = false;
  if (grp == 0)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (r0 + 8 * i < nrows) again |= store_rows<HD>(row_ptr_w<float>(p.dq, b, h, q0 + r0 + 8 * i), acc, i, t, p.scale);
  // rows that are not finite once more (win_rows.cuh)
  if (!__syncthreads_or(again)) return;
  const KeyRows<float> keys{p.k, p.v, b, kvh, nullptr, 0, 0, 0};
  for (int r = threadIdx.x >> 5; r < nrows; r += BWD_THREADS / 32) {
    const int q = q0 + r;
    const int64_t o = ((int64_t)b * p.Hq + h) * p.Npad + q;
    const RowView view{kt, q, 0, kt.count, p.window, p.sinks, p.N};
    mend_dq_row<float, HD, BT>(keys, view, row_ptr<float>(p.q, b, h, q), row_ptr<float>(p.g, b, h, q),
                               row_ptr_w<float>(p.dq, b, h, q), p.c, p.lse2[o], p.dsum[o], p.scale);
  }
}

template <int HD>
__global__ void __launch_bounds__(BWD_THREADS, 1) win_bwd_dkv_f32_kernel(F32Bwd p) {
  constexpr int PA = Pitch<HD>::along, PD = Pitch<HD>::down;
  extern __shared__ float sm[];
  const int grp = threadIdx.x / GROUP, tid = threadIdx.x % GROUP, warp = tid >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3, r0 = 16 * warp + g;
  float* sK = sm;
  float* sV = sK + BT * PA;
  float* sQ = sV + BT * PA + grp * 2 * BT * PD;  // read along (logits) and down (dK, dV)
  float* sG = sQ + BT * PD;
  const int plane = (int)blockIdx.x % p.Hkv + (int)blockIdx.y * p.Hkv;
  const Chunk ch = find_chunk<BT>((int)blockIdx.x / p.Hkv, p.cut, p.L, p.grp, p.N, p.window, p.sinks);
  const int b = plane / p.Hkv, kvh = plane % p.Hkv;
  const int u0 = ch.kt * BT, nq = query_tiles_of<BT>(ch.kt, p.N, p.window, p.sinks);
  const int first = ch.idx * p.L, last = min(first + p.L, nq * p.grp);
  auto key = [&](const TensorRef& x) {
    return [&, x](int r) -> const float* { return u0 + r < p.N ? row_ptr<float>(x, b, kvh, u0 + r) : nullptr; };
  };
  copy_rows<HD, PA>(sK, p.q.p, threadIdx.x, BWD_THREADS, key(p.k));
  copy_rows<HD, PA>(sV, p.q.p, threadIdx.x, BWD_THREADS, key(p.v));
  allow_ahead();
  ahead_wait();
  float dk[HD / 8][4], dv[HD / 8][4];
#pragma unroll
  for (int n = 0; n < HD / 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) dk[n][i] = dv[n][i] = 0.f;
  copies_done();
  __syncthreads();
  for (int s = first + grp; s < last; s += 2) {
    const int h = kvh * p.grp + s / nq, q0 = (ch.kt + s % nq) * BT;
    auto query = [&](const TensorRef& x) {
      return [&, x](int r) -> const float* { return q0 + r < p.N ? row_ptr<float>(x, b, h, q0 + r) : nullptr; };
    };
    copy_rows<HD, PD>(sQ, p.q.p, tid, GROUP, query(p.q));
    copy_rows<HD, PD>(sG, p.q.p, tid, GROUP, query(p.g));
    const float* nl = p.lse2 + ((int64_t)b * p.Hq + h) * p.Npad + q0 + 2 * t;  // -lse2, -D of columns 2t, 2t + 1
    const float* nd = p.dsum + ((int64_t)b * p.Hq + h) * p.Npad + q0 + 2 * t;
    copies_done();
    group_sync(grp);
#pragma unroll 1
    for (int c0 = 0; c0 < BT; c0 += 32) {
      float x[4][4], y[4][4];
      const int k0 = u0 + 16 * warp, t0 = q0 + c0;  // 16 keys, 32 queries
      if (k0 > t0 + 31 || (k0 + 15 <= t0 - p.window && k0 >= p.sinks)) continue;
      logits<HD, PA, PD>(x, sK + 16 * warp * PA, sQ + c0 * PD, g, t);
      logits<HD, PA, PD>(y, sV + 16 * warp * PA, sG + c0 * PD, g, t);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float2 l2 = *reinterpret_cast<const float2*>(nl + c0 + 8 * n), d2 = *reinterpret_cast<const float2*>(nd + c0 + 8 * n);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t vis = visible_queries(u0 + r0 + 8 * i, q0 + c0, p.window, p.sinks) >> (2 * t);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = 2 * i + e;
            const float pv = keep(vis, 8 * n + e, exp2f(fmaf(x[n][k], p.c, e ? l2.y : l2.x)), 0.f);
            x[n][k] = pv;
            y[n][k] = keep(vis, 8 * n + e, pv * (y[n][k] + (e ? d2.y : d2.x)), 0.f);
          }
        }
      }
      weighted<HD, PD>(dv, x, sG + c0 * PD, g, t);
      weighted<HD, PD>(dk, y, sQ + c0 * PD, g, t);
    }
    group_sync(grp);  // Q and g are read
  }
  add_groups<HD>(dk, sV + BT * PA, grp, r0, t);
  add_groups<HD>(dv, sV + BT * PA, grp, r0, t);
  // row `r` of the key tile in the chunk's partials
  auto partial = [&](int r) { return p.part + ((size_t)plane * p.partials + ch.slot + ch.idx) * (2 * BT * HD) + r * HD; };
  bool again = false;
  if (grp == 0)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int u = u0 + r0 + 8 * i;
      if (u >= p.N) continue;
      if (ch.n == 1) {
        again |= store_rows<HD>(row_ptr_w<float>(p.dk, b, kvh, u), dk, i, t, p.scale);
        again |= store_rows<HD>(row_ptr_w<float>(p.dv, b, kvh, u), dv, i, t, 1.0f);
      } else {
        float* base = partial(r0 + 8 * i);
        again |= store_rows<HD>(base, dk, i, t, 1.0f);
        again |= store_rows<HD>(base + BT * HD, dv, i, t, 1.0f);
      }
    }
  // rows that are not finite once more (win_rows.cuh)
  if (!__syncthreads_or(again)) return;
  const QueryView view{p.q, p.g, p.lse2, p.dsum, b, p.Hq, kvh * p.grp, ch.kt, nq, first, last, p.N, p.Npad, p.window, p.sinks};
  for (int r = threadIdx.x >> 5; r < BT && u0 + r < p.N; r += BWD_THREADS / 32) {
    const int u = u0 + r;
    float* part = ch.n == 1 ? nullptr : partial(r);
    mend_dkv_row<float, HD, BT>(view, u, row_ptr<float>(p.k, b, kvh, u), row_ptr<float>(p.v, b, kvh, u), row_ptr_w<float>(p.dk, b, kvh, u),
                                row_ptr_w<float>(p.dv, b, kvh, u), part, part == nullptr ? nullptr : part + BT * HD, p.c, p.scale);
  }
}

// Joins the chunks of one key tile in order: grid (key tiles that may be cut, planes, parts of a tile's rows).  Bound by
// latency: 6 to 7 us for the one sink tile of 8 kv heads (18 MB of partials in fp32 for 14 tiles: 10 us).
template <typename T, int HD, int BTJ>
__global__ void __launch_bounds__(256)
    win_kvjoin_kernel(const float* part, TensorRef dk, TensorRef dv, int Hkv, int grp, int N, int L, int partials,
                      int window, int sinks, float scale) {
  const int kt = blockIdx.x, plane = blockIdx.y, b = plane / Hkv, kvh = plane % Hkv;
  auto chunks_of = [&](int k) {
    return (int)(((long long)query_tiles_of<BTJ>(k, N, window, sinks) * grp + L - 1) / L);
  };
  const int n = chunks_of(kt);
  allow_ahead();
  ahead_wait();
  if (n == 1) return;
  __shared__ int slot_sh;
  if (threadIdx.x < 32) {
    int s = 0;
    for (int k = threadIdx.x; k < kt; k += 32) {
      const int c = chunks_of(k);
      s += c > 1 ? c : 0;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x == 0) slot_sh = s;
  }
  __syncthreads();
  const float* base = part + ((size_t)plane * partials + slot_sh) * (2 * BTJ * HD);
  // blockIdx.z cuts the tile's rows
  const int rows = BTJ / gridDim.z, r0 = blockIdx.z * rows;
  for (int e = threadIdx.x; e < rows * HD / 4; e += 256) {
    const int r = r0 + e / (HD / 4), c = (e % (HD / 4)) * 4, u = kt * BTJ + r;
    if (u >= N) continue;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), v = a;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float* q = base + (size_t)i * (2 * BTJ * HD) + r * HD + c;
      const float4 x = *reinterpret_cast<const float4*>(q), y = *reinterpret_cast<const float4*>(q + BTJ * HD);
      a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
      v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
    }
    T* ok = row_ptr_w<T>(dk, b, kvh, u) + c;
    T* ov = row_ptr_w<T>(dv, b, kvh, u) + c;
    ok[0] = from_f32<T>(a.x * scale);
    ok[1] = from_f32<T>(a.y * scale);
    ok[2] = from_f32<T>(a.z * scale);
    ok[3] = from_f32<T>(a.w * scale);
    ov[0] = from_f32<T>(v.x);
    ov[1] = from_f32<T>(v.y);
    ov[2] = from_f32<T>(v.z);
    ov[3] = from_f32<T>(v.w);
  }
}

template <typename K>
cudaError_t set_smem(K kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int HD>
cudaError_t fwd_t(const WinDims& D, const WinFwdArgs& a, cudaStream_t st) {
  F32Params p{};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.h = a.h;
  p.lse = a.lse;
  p.Hq = D.Hq;
  p.g = D.g;
  p.N = D.N;
  p.window = D.window;
  p.sinks = D.sinks;
  p.NT = (D.N + BT - 1) / BT;
  p.c = D.scale * kLog2e;
  auto kern = win_fwd_f32_kernel<HD, false>;
  cudaError_t e = set_smem(kern, Fwd<HD>::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)((int64_t)p.NT * D.B * D.Hq), Fwd<HD>::THREADS, Fwd<HD>::SMEM, st>>>(p);
  count_launches(1);
  return cudaGetLastError();
}

template <int HD>
cudaError_t bwd_t(const WinDims& D, const WinBwdArgs& a, cudaStream_t st) {
  cudaError_t e = launch_win_bwd_pre(D, a, st);
  if (e != cudaSuccess) return e;
  const WinBwdLayout L = win_bwd_layout(D);
  const ChunkPlan cp = chunk_plan<BT>(D, kBwdChunks, kMinSteps);
  char* ws = static_cast<char*>(a.ws);
  F32Bwd p{};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.g = a.g;
  p.dq = a.dq;
  p.dk = a.dk;
  p.dv = a.dv;
  p.lse2 = reinterpret_cast<const float*>(ws + L.lse2);
  p.dsum = reinterpret_cast<const float*>(ws + L.dsum);
  p.part = reinterpret_cast<float*>(ws + L.part);
  p.Hq = D.Hq;
  p.Hkv = D.Hkv;
  p.grp = D.g;
  p.N = D.N;
  p.Npad = L.Npad;
  p.window = D.window;
  p.sinks = D.sinks;
  p.NT = cp.NT;
  p.L = cp.L;
  p.partials = cp.partials;
  p.cut = cp.cut;
  p.c = D.scale * kLog2e;
  p.scale = D.scale;
  auto dkv = win_bwd_dkv_f32_kernel<HD>;
  if ((e = set_smem(dkv, bwd_smem<HD>())) != cudaSuccess) return e;
  if ((e = launch_ahead(dkv, dim3(cp.chunks * D.Hkv, D.B), BWD_THREADS, bwd_smem<HD>(), st, p)) != cudaSuccess) return e;
  if ((e = launch_win_kvjoin<BT>(D, a, cp, p.part, st)) != cudaSuccess) return e;
  auto dq = win_bwd_dq_f32_kernel<HD>;
  if ((e = set_smem(dq, bwd_smem<HD>())) != cudaSuccess) return e;
  return launch_ahead(dq, dim3((unsigned)((int64_t)cp.NT * D.B * D.Hq)), BWD_THREADS, bwd_smem<HD>(), st, p);
}

template <typename T, int HD>
cudaError_t pre_t(const WinDims& D, const WinBwdArgs& a, cudaStream_t st) {
  const WinBwdLayout L = win_bwd_layout(D);
  char* ws = static_cast<char*>(a.ws);
  constexpr int per = 8 * 4 * (32 / (HD / Vec16<T>::kN));  // rows of a CTA
  win_bwd_pre_kernel<T, HD><<<dim3((L.Npad + per - 1) / per, D.B * D.Hq), 256, 0, st>>>(
      a.h, a.g, a.lse, reinterpret_cast<float*>(ws + L.lse2), reinterpret_cast<float*>(ws + L.dsum), D.Hq, D.N, L.Npad);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T, int HD, int BTJ>
cudaError_t join_t(const WinDims& D, const WinBwdArgs& a, const ChunkPlan& p, const float* part, cudaStream_t st) {
  return launch_ahead(win_kvjoin_kernel<T, HD, BTJ>, dim3(p.cut, D.B * D.Hkv, 8), 256, 0, st, part, a.dk, a.dv, D.Hkv, D.g,
                      D.N, p.L, p.partials, D.window, D.sinks, D.scale);
}

template <int HD>
cudaError_t paged_t(const PagedDims& D, const PagedArgs& a, cudaStream_t st) {
  F32Params p{};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.h = a.h;
  p.lse = a.lse;
  p.Hq = D.Hq;
  p.g = D.g;
  p.window = D.window;
  p.sinks = D.sinks;
  p.c = D.scale * kLog2e;
  p.table = a.table;
  p.page = D.page;
  p.num_pages = D.num_pages;
  p.max_pages = D.max_pages;
  p.T = D.T;
  const int TI = BT / D.g;
  p.batch = Batch{a.q_start, a.kv_len, D.seqs, D.T, D.max_pages * D.page, TI, D.window, D.sinks, D.Hkv};
  p.part = static_cast<float*>(a.ws);
  auto kern = win_fwd_f32_kernel<HD, true>;
  cudaError_t e = set_smem(kern, Fwd<HD>::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<kPagedCtas, Fwd<HD>::THREADS, Fwd<HD>::SMEM, st>>>(p);
  count_launches(1);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_paged_join<BT, BT>(D, a, kPagedCtas, TI, st);
}

}  // namespace

cudaError_t launch_win_fwd_f32(const WinDims& D, const WinFwdArgs& a, cudaStream_t st) {
  return D.d == 64 ? fwd_t<64>(D, a, st) : fwd_t<128>(D, a, st);
}
cudaError_t launch_win_bwd_pre(const WinDims& D, const WinBwdArgs& a, cudaStream_t st) {
  if (D.dtype == SSA_BF16) return D.d == 64 ? pre_t<__nv_bfloat16, 64>(D, a, st) : pre_t<__nv_bfloat16, 128>(D, a, st);
  return D.d == 64 ? pre_t<float, 64>(D, a, st) : pre_t<float, 128>(D, a, st);
}
cudaError_t launch_win_bwd_f32(const WinDims& D, const WinBwdArgs& a, cudaStream_t st) {
  return D.d == 64 ? bwd_t<64>(D, a, st) : bwd_t<128>(D, a, st);
}
cudaError_t launch_paged_f32(const PagedDims& D, const PagedArgs& a, cudaStream_t st) {
  return D.d == 64 ? paged_t<64>(D, a, st) : paged_t<128>(D, a, st);
}

template <int BTJ>
cudaError_t launch_win_kvjoin(const WinDims& D, const WinBwdArgs& a, const ChunkPlan& p, const float* part,
                              cudaStream_t st) {
  if (p.partials == 0) return cudaSuccess;
  using T = std::conditional_t<BTJ == 128, __nv_bfloat16, float>;  // tiles of 128 tokens are the bf16 kernels'
  return D.d == 64 ? join_t<T, 64, BTJ>(D, a, p, part, st) : join_t<T, 128, BTJ>(D, a, p, part, st);
}
template cudaError_t launch_win_kvjoin<64>(const WinDims&, const WinBwdArgs&, const ChunkPlan&, const float*, cudaStream_t);
template cudaError_t launch_win_kvjoin<128>(const WinDims&, const WinBwdArgs&, const ChunkPlan&, const float*, cudaStream_t);

WinBwdLayout win_bwd_layout(const WinDims& D) {
  WinBwdLayout L{};
  L.Npad = (D.N + 127) / 128 * 128;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = (size_t)D.B * D.Hq * L.Npad;
  size_t o = 0;
  L.lse2 = o;
  o = up(o + rows * 4);
  L.dsum = o;
  o = up(o + rows * 4);
  L.part = o;
  const int tile = D.dtype == SSA_BF16 ? 128 : BT;
  const ChunkPlan p = D.dtype == SSA_BF16 ? chunk_plan<128>(D, kBwdChunks, kTcMinSteps) : chunk_plan<BT>(D, kBwdChunks, kMinSteps);
  o = up(o + (size_t)D.B * D.Hkv * p.partials * 2 * tile * D.d * 4);
  L.bytes = o;
  return L;
}

size_t paged_ws_bytes(const PagedDims& D) {
  return ((size_t)2 * kPagedCtas * partial_floats(BT, D.d) * 4 + 255) / 256 * 256;
}

}  // namespace ssa
