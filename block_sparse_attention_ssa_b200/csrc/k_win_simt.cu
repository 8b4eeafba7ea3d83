// Window attention with sinks and paged attention in fp32 on CUDA cores, and the
// preprocess and the join of the backward for both types.
//
// Mathematics: the online softmax over the visible keys (base 2, scale folded in)
// and, backward, p = 2^(x c - lse2), dx = p (g.v - D), dQ = scale dx K,
// dK = scale dx^T Q, dV = p^T g.  fp32 arithmetic throughout, because no tensor-core
// input type holds fp32 values.
//
// Tiles: 64 queries by 64 keys, 256 threads, thread (tx, ty) owns queries 4 ty .. and
// keys tx + 16 j: a step of four head dims is 8 16-byte shared loads (12 wavefronts) for
// 64 multiply-adds a thread, so the FMA pipe, not shared memory, sets the pace.
#include "win_common.cuh"

#include <type_traits>

#include "sm100_ptx.cuh"

namespace ssa {
namespace {

using sm100::fma2;

constexpr int BT = 64;
constexpr int GROUP = 256;          // threads on one 64 x 64 tile
constexpr int THREADS = 2 * GROUP;  // two groups in a CTA
constexpr int SP = BT + 4;  // row pitch of the P tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// CTAs of one paged call, one per SM; units are worth a CTA from two on.
constexpr int kPagedCtas = 148;
constexpr int kMinUnits = 2;
// Steps of a backward chunk at least: a 64 x 64 step takes some 9 us of a CTA, a partial's round trip less.
constexpr int kMinSteps = 2;

template <int HD>
struct Pitch {
  static constexpr int v = HD + 4;
};

struct SimtParams {
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

// A 64-row tile on its way through registers, so that its loads are in flight while the tile before is used; a
// null row pointer gives zeros.
template <int HD, int TH>
struct TileRegs {  // by the TH threads of a group or of the CTA
  static constexpr int PER = HD / 4, N = BT * PER / TH;
  float4 v[N];
  template <typename F>
  __device__ __forceinline__ void fetch(F row) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = threadIdx.x % TH + i * TH;
      const float* p = row(e / PER);
      v[i] = p != nullptr ? *reinterpret_cast<const float4*>(p + (e % PER) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void put(float* dst) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = threadIdx.x % TH + i * TH;
      *reinterpret_cast<float4*>(dst + (e / PER) * Pitch<HD>::v + (e % PER) * 4) = v[i];
    }
  }
};

// s[i][j] = A[4 ty + i] . B[tx + 16 j], even and odd head dims in the two halves of a packed multiply-add.
template <int HD>
__device__ __forceinline__ void dots(const float* A, const float* B, int tx, int ty, float (&s)[4][4]) {
  constexpr int P = Pitch<HD>::v;
  float2 t[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) t[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < HD; k += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * P + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * P + k);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        t[i][j] = fma2(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), t[i][j]);
        t[i][j] = fma2(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), t[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = t[i][j].x + t[i][j].y;
}

// acc[i][.] += sum_u W[4 ty + i][u] X[u][.]; columns 4 tx + 64 q + 0..3.
template <int HD>
__device__ __forceinline__ void weighted(const float* W, const float* X, int tx, int ty, float (&acc)[4][HD / 16]) {
#pragma unroll 2
  for (int u = 0; u < BT; u += 4) {
    float w[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 t = *reinterpret_cast<const float4*>(W + (4 * ty + i) * SP + u);
      w[i][0] = t.x;
      w[i][1] = t.y;
      w[i][2] = t.z;
      w[i][3] = t.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int q = 0; q < HD / 64; ++q) {
        const float4 x = *reinterpret_cast<const float4*>(X + (u + e) * Pitch<HD>::v + 64 * q + 4 * tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 ww = make_float2(w[i][e], w[i][e]);
          const float2 lo = fma2(ww, make_float2(x.x, x.y), make_float2(acc[i][4 * q], acc[i][4 * q + 1]));
          const float2 hi = fma2(ww, make_float2(x.z, x.w), make_float2(acc[i][4 * q + 2], acc[i][4 * q + 3]));
          acc[i][4 * q] = lo.x;
          acc[i][4 * q + 1] = lo.y;
          acc[i][4 * q + 2] = hi.x;
          acc[i][4 * q + 3] = hi.y;
        }
      }
  }
}

template <int HD>
__device__ __forceinline__ void store_row(float* dst, const float* acc, int tx, float mul) {
#pragma unroll
  for (int q = 0; q < HD / 64; ++q)
    *reinterpret_cast<float4*>(dst + 64 * q + 4 * tx) =
        make_float4(acc[4 * q] * mul, acc[4 * q + 1] * mul, acc[4 * q + 2] * mul, acc[4 * q + 3] * mul);
}

// Q, then each group's tile (K, then V) and weights.
template <int HD>
constexpr size_t fwd_smem() {
  return (size_t)(3 * BT * Pitch<HD>::v + 2 * BT * SP) * 4;
}

__device__ __forceinline__ void group_sync(int grp) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(GROUP) : "memory");
}

// ================================================================ forward
// The two groups of a CTA take its key tiles in turn, each with its own online softmax, and join them at the end:
// few rows fill the GPU's warps too (one group took 37 us at N = 1021, 8 heads and sequences, window 200).
template <int HD, bool PAGED>
__global__ void __launch_bounds__(THREADS, 1) win_fwd_simt_kernel(SimtParams p) {
  extern __shared__ float sm[];
  float* sQ = sm;
  const int grp = threadIdx.x / GROUP, tid = threadIdx.x % GROUP, tx = tid & 15, ty = tid >> 4;
  float* sX = sQ + (1 + grp) * BT * Pitch<HD>::v;  // K, then V
  float* sP = sQ + 3 * BT * Pitch<HD>::v + grp * BT * SP;
  __shared__ Place sh_place;
  __shared__ int sh_left;
  __shared__ float sh_m[BT], sh_l[BT];

  Place at{0, 0, 0, 0};
  int left = 1;
  if (PAGED) {
    if (threadIdx.x < 32) {
      const long long U = p.batch.total<BT>();
      const long long per = share(U, (int)gridDim.x, kMinUnits);
      const long long u0 = per * blockIdx.x;
      const long long n = u0 < U ? min(per, U - u0) : 0;
      if (n > 0) at = p.batch.locate<BT>(u0);
      if (threadIdx.x == 0) {
        sh_place = at;
        sh_left = (int)n;
      }
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be brought up
    at = sh_place;
    left = sh_left;
  }

  for (int seg = 0; left > 0; ++seg) {
    // ---- the item
    int b, head0, q0row, kvh, nrows, p0, per_tok, i0 = 0, units, take, len, part_rows = 0;
    Seq s{};
    KeyTiles kt;
    if (PAGED) {
      b = at.b;
      s = load_seq(p.batch.q_start, p.batch.kv_len, b, p.T, p.batch.cap);
      i0 = at.run * p.batch.TI;
      const int toks = min(p.batch.TI, s.n - i0);
      kvh = at.kvh;
      head0 = kvh * p.g;
      per_tok = p.g;
      nrows = toks * p.g;
      q0row = s.q0 + i0;
      p0 = s.len - s.n + i0;
      len = s.len;
      kt = run_tiles<BT>(s, i0, p.batch.TI, p.window, p.sinks);
      units = max(1, kt.count);
      take = min(left, units - at.off);
      part_rows = take < units ? nrows : 0;
    } else {
      const int planes = (int)(gridDim.x / p.NT);
      const int plane = (int)blockIdx.x % planes, qt = p.NT - 1 - (int)blockIdx.x / planes;
      b = plane / p.Hq;
      head0 = plane % p.Hq;
      kvh = head0 / p.g;
      per_tok = 1;
      q0row = p0 = qt * BT;
      nrows = min(BT, p.N - p0);
      len = p.N;
      kt = key_tiles<BT>(p0, p0 + nrows - 1, p.window, p.sinks);
      units = take = kt.count;
    }
    auto tok_of = [&](int r) { return PAGED ? r / per_tok : r; };
    auto head_of = [&](int r) { return PAGED ? head0 + r % per_tok : head0; };
    TileRegs<HD, GROUP> regs;
    if (grp == 0) {
      regs.fetch([&](int r) -> const float* {
        return r < nrows ? row_ptr<float>(p.q, PAGED ? 0 : b, head_of(r), q0row + tok_of(r)) : nullptr;
      });
      regs.put(sQ);
    }

    float acc[4][HD / 16], m[4], l[4];
    int pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = kNegInf;
      l[i] = 0.f;
      pos[i] = 4 * ty + i < nrows ? p0 + tok_of(4 * ty + i) : -1;
#pragma unroll
      for (int c = 0; c < HD / 16; ++c) acc[i][c] = 0.f;
    }
    const int pmax = p0 + tok_of(nrows - 1), lo_min = p0 - p.window + 1;

    // A key that no row of the item sees is not read (its memory may hold anything).
    auto keys = [&](const TensorRef& t, int j) {
      const int u0 = kt.tile(j) * BT;
      return [&, t, u0](int r) -> const float* {
        const int u = u0 + r;
        if (u > pmax || u >= len || (u < lo_min && u >= p.sinks)) return nullptr;
        if (!PAGED) return row_ptr<float>(t, b, kvh, u);
        const int pg = p.table[(int64_t)b * p.max_pages + u / p.page];
        return (unsigned)pg < (unsigned)p.num_pages ? row_ptr<float>(t, pg, kvh, u % p.page) : nullptr;
      };
    };
    const int end = min(at.off + take, kt.count);
    if (at.off + grp < end) regs.fetch(keys(p.k, at.off + grp));
    __syncthreads();  // Q is there
    for (int j = at.off + grp; j < end; j += 2) {
      const int u0 = kt.tile(j) * BT;
      group_sync(grp);
      regs.put(sX);
      group_sync(grp);
      regs.fetch(keys(p.v, j));
      float x[4][4];
      dots<HD>(sQ, sX, tx, ty, x);
      bool held[4];
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        held[jj] = true;
        if (PAGED) {
          const int u = u0 + tx + 16 * jj;
          held[jj] = u < len && (unsigned)p.table[(int64_t)b * p.max_pages + u / p.page] < (unsigned)p.num_pages;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = kNegInf;
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int u = u0 + tx + 16 * jj;
          const bool see = held[jj] && u <= pos[i] && (u > pos[i] - p.window || u < p.sinks);
          x[i][jj] = see ? x[i][jj] * p.c : kNegInf;
          mx = fmaxf(mx, x[i][jj]);
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m[i], mx);
        const float ref = mn == kNegInf ? 0.f : mn;
        const float f = exp2f(m[i] - ref);
        float sum = 0.f;
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const float e = exp2f(x[i][jj] - ref);
          sum += e;
          sP[(4 * ty + i) * SP + tx + 16 * jj] = e;
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = l[i] * f + sum;
        m[i] = mn;
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) acc[i][c] *= f;
      }
      group_sync(grp);
      regs.put(sX);
      group_sync(grp);
      if (j + 2 < end) regs.fetch(keys(p.k, j + 2));
      weighted<HD>(sP, sX, tx, ty, acc);
    }

    // ---- join of the groups' softmaxes
    if (grp == 1) {
      group_sync(1);  // sX is read to the end
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        store_row<HD>(sX + (4 * ty + i) * Pitch<HD>::v, acc[i], tx, 1.0f);
        if (tx == 0) {
          sh_m[4 * ty + i] = m[i];
          sh_l[4 * ty + i] = l[i];
        }
      }
    }
    __syncthreads();
    if (grp == 0) {
      const float* other = sX + BT * Pitch<HD>::v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        const float m1 = sh_m[r], mn = fmaxf(m[i], m1), ref = mn == kNegInf ? 0.f : mn;
        const float f0 = exp2f(m[i] - ref), f1 = exp2f(m1 - ref);
        l[i] = l[i] * f0 + sh_l[r] * f1;
        m[i] = mn;
#pragma unroll
        for (int q = 0; q < HD / 64; ++q) {
          const float4 o = *reinterpret_cast<const float4*>(other + r * Pitch<HD>::v + 64 * q + 4 * tx);
          acc[i][4 * q] = acc[i][4 * q] * f0 + o.x * f1;
          acc[i][4 * q + 1] = acc[i][4 * q + 1] * f0 + o.y * f1;
          acc[i][4 * q + 2] = acc[i][4 * q + 2] * f0 + o.z * f1;
          acc[i][4 * q + 3] = acc[i][4 * q + 3] * f0 + o.w * f1;
        }
      }
    }
    // ---- epilogue
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * ty + i;
      if (r >= nrows || grp == 1) continue;
      if (PAGED && part_rows) {
        float* base = p.part + (size_t)(2 * blockIdx.x + (seg ? 1 : 0)) * partial_floats(BT, HD);
#pragma unroll
        for (int q = 0; q < HD / 64; ++q)
          *reinterpret_cast<float4*>(base + r * HD + 64 * q + 4 * tx) =
              make_float4(acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]);
        if (tx == 0) {
          base[BT * HD + r] = m[i];
          base[BT * HD + BT + r] = l[i];
        }
        continue;
      }
      const float inv = l[i] == 0.f ? 0.f : 1.0f / l[i];
      store_row<HD>(row_ptr_w<float>(p.h, PAGED ? 0 : b, head_of(r), q0row + tok_of(r)), acc[i], tx, inv);
      if (tx == 0) {
        const int64_t o = PAGED ? (int64_t)head_of(r) * p.T + q0row + tok_of(r)
                                : ((int64_t)b * p.Hq + head0) * p.N + q0row + r;
        p.lse[o] = l[i] == 0.f ? kNegInf : (m[i] + log2f(l[i])) * kLn2;
      }
    }
    if (!PAGED) break;
    // ---- the next item
    left -= take;
    if (left <= 0) break;
    at.off = 0;
    if (++at.kvh == p.batch.Hkv) {
      at.kvh = 0;
      ++at.run;
      while (at.b < p.batch.seqs) {
        s = load_seq(p.batch.q_start, p.batch.kv_len, at.b, p.T, p.batch.cap);
        if (at.run * p.batch.TI < s.n) break;
        at.run = 0;
        ++at.b;
      }
      if (at.b >= p.batch.seqs) break;
    }
    __syncthreads();  // sQ, sX and sP are read to the end
  }
}

// ================================================================ backward
// -D_t = -(g_t . h_t) and -lse in base 2, rows padded to 128 tokens.  Bound by reading h and g: a row is LPR
// lanes of 16 bytes, and a warp has four rows' loads of each in flight per lane group.
template <typename T, int HD>
__global__ void __launch_bounds__(256) win_bwd_pre_kernel(TensorRef h, TensorRef g, const float* lse, float* lse2,
                                                          float* dsum, int Hq, int N, int Npad) {
  constexpr int V = Vec16<T>::kN, LPR = HD / V, RPW = 32 / LPR, U = 4;
  const int lane = threadIdx.x & 31, c = lane % LPR * V;
  const int bh = blockIdx.y, b = bh / Hq, hd = bh % Hq;
  const int t0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * (RPW * U) + lane / LPR;
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

struct SimtBwd {
  TensorRef q, k, v, g, dq, dk, dv;
  const float* lse2;
  const float* dsum;
  float* part;
  int Hq, Hkv, grp, N, Npad, window, sinks, NT, L, partials, cut;
  float c, scale;
};

// The first group forms the weights, the second dP, side by side (twice the warps
// for the same tiles; one group of 256 took 165 us for dkv and 77 us for dq at N = 1000, 8 heads, d = 128).
// The next step's tiles are fetched into registers while this one is computed.
template <int HD>
constexpr size_t bwd_smem() {
  return (size_t)(4 * BT * Pitch<HD>::v + 2 * BT * SP) * 4;
}

__device__ __forceinline__ void put4x4(float* P, const float (&x)[4][4], int tx, int ty) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) P[(4 * ty + i) * SP + tx + 16 * jj] = x[i][jj];
}

template <int HD>
__global__ void __launch_bounds__(THREADS, 1) win_bwd_dq_simt_kernel(SimtBwd p) {
  extern __shared__ float sm[];
  float* sQ = sm;
  float* sG = sQ + BT * Pitch<HD>::v;
  float* sK = sG + BT * Pitch<HD>::v;
  float* sV = sK + BT * Pitch<HD>::v;
  float* sP = sV + BT * Pitch<HD>::v;
  float* sS = sP + BT * SP;
  const int grp = threadIdx.x >> 8, tid = threadIdx.x & 255, tx = tid & 15, ty = tid >> 4;
  const int planes = (int)(gridDim.x / p.NT);
  const int plane = (int)blockIdx.x % planes, qt = p.NT - 1 - (int)blockIdx.x / planes;
  const int b = plane / p.Hq, h = plane % p.Hq, kvh = h / p.grp;
  const int q0 = qt * BT, nrows = min(BT, p.N - q0);
  const KeyTiles kt = key_tiles<BT>(q0, q0 + nrows - 1, p.window, p.sinks);
  TileRegs<HD, THREADS> ra, rb;
  auto query = [&](const TensorRef& t) {
    return [&, t](int r) -> const float* { return r < nrows ? row_ptr<float>(t, b, h, q0 + r) : nullptr; };
  };
  auto key = [&](const TensorRef& t, int j) {
    const int u0 = kt.tile(j) * BT;
    return [&, t, u0](int r) -> const float* { return u0 + r < p.N ? row_ptr<float>(t, b, kvh, u0 + r) : nullptr; };
  };
  ra.fetch(query(p.q));
  rb.fetch(query(p.g));
  ra.put(sQ);
  rb.put(sG);
  ra.fetch(key(p.k, 0));
  rb.fetch(key(p.v, 0));
  constexpr int CT = HD / 32;  // columns of a thread: CT tx + HD/2 grp ..
  const int col = CT * tx + HD / 2 * grp;
  float st[4], acc[4][CT];  // st: -lse2 (first group), -D (second)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t o = ((int64_t)b * p.Hq + h) * p.Npad + q0 + 4 * ty + i;
    st[i] = grp ? p.dsum[o] : p.lse2[o];
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[i][c] = 0.f;
  }
  for (int j = 0; j < kt.count; ++j) {
    const int u0 = kt.tile(j) * BT;
    __syncthreads();
    ra.put(sK);
    rb.put(sV);
    __syncthreads();
    if (j + 1 < kt.count) {
      ra.fetch(key(p.k, j + 1));
      rb.fetch(key(p.v, j + 1));
    }
    float x[4][4];
    dots<HD>(grp ? sG : sQ, grp ? sV : sK, tx, ty, x);
    if (grp == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int u = u0 + tx + 16 * jj, t = q0 + 4 * ty + i;
          const bool see = u <= t && (t - u < p.window || u < p.sinks);
          x[i][jj] = see ? exp2f(fmaf(x[i][jj], p.c, st[i])) : 0.f;
        }
      put4x4(sP, x, tx, ty);
    }
    __syncthreads();
    if (grp == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const float pv = sP[(4 * ty + i) * SP + tx + 16 * jj];
          x[i][jj] = pv != 0.f ? pv * (x[i][jj] + st[i]) : 0.f;
        }
      put4x4(sS, x, tx, ty);
    }
    __syncthreads();
#pragma unroll 2
    for (int u = 0; u < BT; u += 4) {
      float w[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 t = *reinterpret_cast<const float4*>(sS + (4 * ty + i) * SP + u);
        w[i][0] = t.x;
        w[i][1] = t.y;
        w[i][2] = t.z;
        w[i][3] = t.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* kr = sK + (u + e) * Pitch<HD>::v + col;
#pragma unroll
        for (int c = 0; c < CT; c += 2) {
          const float2 k2 = *reinterpret_cast<const float2*>(kr + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a2 = fma2(make_float2(w[i][e], w[i][e]), k2, make_float2(acc[i][c], acc[i][c + 1]));
            acc[i][c] = a2.x;
            acc[i][c + 1] = a2.y;
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (4 * ty + i < nrows) {
      float* dst = row_ptr_w<float>(p.dq, b, h, q0 + 4 * ty + i) + col;
#pragma unroll
      for (int c = 0; c < CT; c += 2) *reinterpret_cast<float2*>(dst + c) = make_float2(acc[i][c] * p.scale, acc[i][c + 1] * p.scale);
    }
}

template <int HD>
__global__ void __launch_bounds__(THREADS, 1) win_bwd_dkv_simt_kernel(SimtBwd p) {
  extern __shared__ float sm[];
  float* sK = sm;
  float* sV = sK + BT * Pitch<HD>::v;
  float* sQ = sV + BT * Pitch<HD>::v;
  float* sG = sQ + BT * Pitch<HD>::v;
  float* sP = sG + BT * Pitch<HD>::v;
  float* sS = sP + BT * SP;
  const int grp = threadIdx.x >> 8, tid = threadIdx.x & 255, tx = tid & 15, ty = tid >> 4;
  const int plane = (int)blockIdx.x % p.Hkv + (int)blockIdx.y * p.Hkv;
  const Chunk ch = find_chunk<BT>((int)blockIdx.x / p.Hkv, p.cut, p.L, p.grp, p.N, p.window, p.sinks);
  const int b = plane / p.Hkv, kvh = plane % p.Hkv;
  const int u0 = ch.kt * BT, nq = query_tiles_of<BT>(ch.kt, p.N, p.window, p.sinks);
  const int first = ch.idx * p.L, last = min(first + p.L, nq * p.grp);
  TileRegs<HD, THREADS> ra, rb;
  float nx[4];  // -lse2 (first group) or -D (second) of the next step
  auto key = [&](const TensorRef& t) {
    return [&, t](int r) -> const float* { return u0 + r < p.N ? row_ptr<float>(t, b, kvh, u0 + r) : nullptr; };
  };
  auto fetch = [&](int s) {
    const int h = kvh * p.grp + s / nq, q0 = (ch.kt + s % nq) * BT;
    ra.fetch([&](int r) -> const float* { return q0 + r < p.N ? row_ptr<float>(p.q, b, h, q0 + r) : nullptr; });
    rb.fetch([&](int r) -> const float* { return q0 + r < p.N ? row_ptr<float>(p.g, b, h, q0 + r) : nullptr; });
    const float* row = (grp ? p.dsum : p.lse2) + ((int64_t)b * p.Hq + h) * p.Npad + q0 + tx;
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) nx[jj] = row[16 * jj];
  };
  ra.fetch(key(p.k));
  rb.fetch(key(p.v));
  ra.put(sK);
  rb.put(sV);
  fetch(first);
  float acc[4][HD / 16];  // dV (first group) or dK (second)
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < HD / 16; ++c) acc[i][c] = 0.f;
  for (int s = first; s < last; ++s) {
    const int q0 = (ch.kt + s % nq) * BT;
    float st[4];
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) st[jj] = nx[jj];
    __syncthreads();
    ra.put(sQ);
    rb.put(sG);
    __syncthreads();
    if (s + 1 < last) fetch(s + 1);
    float x[4][4];
    dots<HD>(grp ? sV : sK, grp ? sG : sQ, tx, ty, x);
    if (grp == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int u = u0 + 4 * ty + i, t = q0 + tx + 16 * jj;
          const bool see = u <= t && (t - u < p.window || u < p.sinks);
          x[i][jj] = see ? exp2f(fmaf(x[i][jj], p.c, st[jj])) : 0.f;
        }
      put4x4(sP, x, tx, ty);
    }
    __syncthreads();
    if (grp == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const float pv = sP[(4 * ty + i) * SP + tx + 16 * jj];
          x[i][jj] = pv != 0.f ? pv * (x[i][jj] + st[jj]) : 0.f;
        }
      put4x4(sS, x, tx, ty);
      asm volatile("bar.sync 1, 256;" ::: "memory");  // the second group's own tile
    }
    weighted<HD>(grp ? sS : sP, grp ? sQ : sG, tx, ty, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int u = u0 + 4 * ty + i;
    if (u >= p.N) continue;
    if (ch.n == 1) {
      store_row<HD>(row_ptr_w<float>(grp ? p.dk : p.dv, b, kvh, u), acc[i], tx, grp ? p.scale : 1.0f);
    } else {
      float* base = p.part + ((size_t)plane * p.partials + ch.slot + ch.idx) * (2 * BT * HD) + (grp ? 0 : BT * HD) + (4 * ty + i) * HD;
#pragma unroll
      for (int q = 0; q < HD / 64; ++q)
        *reinterpret_cast<float4*>(base + 64 * q + 4 * tx) =
            make_float4(acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]);
    }
  }
}

// Joins the chunks of one key tile in order: grid (key tiles that may be cut, planes, parts of a tile's rows).
template <typename T, int HD, int BTJ>
__global__ void __launch_bounds__(256)
    win_kvjoin_kernel(const float* part, TensorRef dk, TensorRef dv, int Hkv, int grp, int N, int L, int partials,
                      int window, int sinks, float scale) {
  const int kt = blockIdx.x, plane = blockIdx.y, b = plane / Hkv, kvh = plane % Hkv;
  auto chunks_of = [&](int k) {
    return (int)(((long long)query_tiles_of<BTJ>(k, N, window, sinks) * grp + L - 1) / L);
  };
  const int n = chunks_of(kt);
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
  SimtParams p{};
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
  auto kern = win_fwd_simt_kernel<HD, false>;
  cudaError_t e = set_smem(kern, fwd_smem<HD>());
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)((int64_t)p.NT * D.B * D.Hq), THREADS, fwd_smem<HD>(), st>>>(p);
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
  SimtBwd p{};
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
  auto dkv = win_bwd_dkv_simt_kernel<HD>;
  if ((e = set_smem(dkv, bwd_smem<HD>())) != cudaSuccess) return e;
  dkv<<<dim3(cp.chunks * D.Hkv, D.B), THREADS, bwd_smem<HD>(), st>>>(p);
  count_launches(1);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = launch_win_kvjoin<BT>(D, a, cp, p.part, st)) != cudaSuccess) return e;
  auto dq = win_bwd_dq_simt_kernel<HD>;
  if ((e = set_smem(dq, bwd_smem<HD>())) != cudaSuccess) return e;
  dq<<<(unsigned)((int64_t)cp.NT * D.B * D.Hq), THREADS, bwd_smem<HD>(), st>>>(p);
  count_launches(1);
  return cudaGetLastError();
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
  win_kvjoin_kernel<T, HD, BTJ><<<dim3(p.cut, D.B * D.Hkv, 8), 256, 0, st>>>(
      part, a.dk, a.dv, D.Hkv, D.g, D.N, p.L, p.partials, D.window, D.sinks, D.scale);
  count_launches(1);
  return cudaGetLastError();
}

template <int HD>
cudaError_t paged_t(const PagedDims& D, const PagedArgs& a, cudaStream_t st) {
  SimtParams p{};
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
  auto kern = win_fwd_simt_kernel<HD, true>;
  cudaError_t e = set_smem(kern, fwd_smem<HD>());
  if (e != cudaSuccess) return e;
  kern<<<kPagedCtas, THREADS, fwd_smem<HD>(), st>>>(p);
  count_launches(1);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_paged_join<BT, BT>(D, a, kPagedCtas, TI, kMinUnits, st);
}

}  // namespace

cudaError_t launch_win_fwd_simt(const WinDims& D, const WinFwdArgs& a, cudaStream_t st) {
  return D.d == 64 ? fwd_t<64>(D, a, st) : fwd_t<128>(D, a, st);
}
cudaError_t launch_win_bwd_pre(const WinDims& D, const WinBwdArgs& a, cudaStream_t st) {
  if (D.dtype == SSA_BF16) return D.d == 64 ? pre_t<__nv_bfloat16, 64>(D, a, st) : pre_t<__nv_bfloat16, 128>(D, a, st);
  return D.d == 64 ? pre_t<float, 64>(D, a, st) : pre_t<float, 128>(D, a, st);
}
cudaError_t launch_win_bwd_simt(const WinDims& D, const WinBwdArgs& a, cudaStream_t st) {
  return D.d == 64 ? bwd_t<64>(D, a, st) : bwd_t<128>(D, a, st);
}
cudaError_t launch_paged_simt(const PagedDims& D, const PagedArgs& a, cudaStream_t st) {
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
