// Backward of window attention with sinks on tcgen05 (bf16, d = 64 or 128).
//
// Mathematics: p = 2^(s c - lse2), dP = g V^T, dx = p (dP - D) with D_t = g_t . h_t;
// dV = p^T g, dK = scale dx^T Q, dQ = scale dx K.  Logits, p, dP, dx and all sums are
// fp32; p and dx are rounded to bf16 (half a step each) as operands of the next product.
// -lse2 and -D come from the preprocess in rows padded to 128 tokens; a padding row's -lse2
// is -infinity, which makes its weights zero.
//
// Two kernels of 576 threads, each forming S and dP: a query tile's dQ and a key tile's dK,
// dV have different owners, and joining them through memory costs more than the two extra
// products (a dQ of fp32 additions in L2 moves 64 KB per 128 x 128 tile).  No atomics, and one
// thread issues all products of a CTA: every output has one writer with a fixed order.
// Warps 0-15 compute, 32 rows by 32 columns each, warp 16 loads by TMA, warp 17 issues.
//
//   dkv  a 128-key tile and a chunk of its units (query head, 64 queries) per CTA.  TMEM
//        (512 columns at d = 128): dK, dV, two S^T, two dP^T.  Two groups of eight warps take
//        the units in turn, one turning logits into weights while the other forms gradients,
//        so that the exponentials (16 a cycle and SM) and the tensor core work side by side;
//        with all warps on one 128-wide step they took turns (4000 cycles a 128 x 128 tile).
//        The products go round dV(i), S^T(i+2), dK(i-1), dP^T(i+1); P^T overwrites S^T, dx^T
//        overwrites dP^T, each warp within its own columns.
//   dq   a persistent CTA walks (query head, 128-query tile) items over tiles of 128 keys.
//        TMEM: dQ, two S, dP.  dx overwrites the S it came from, so that dP(j+1) can be formed
//        as soon as dP(j) is read; the products go round dP(j+1), dQ(j), S(j+2), and the warps
//        form the weights of j + 1 meanwhile.
//
// Measured (16384 tokens, 32 heads over 8, d = 128, window 1024, 64 sinks): dkv 530 us, tensor pipe busy 64 % of the time
// (1400 to 1600 cycles a unit, 1280 of them products); dq 437 us, 57 % (exponentials and dx, a chain of 1800
// cycles a tile); with the preprocess (50 us) and the join (7 us) 680 TFLOP/s of the five products that count; seven are formed.
#include "win_rows.cuh"

#include "sm100_ptx.cuh"

namespace ssa {
namespace {

using namespace sm100;
using bf16 = __nv_bfloat16;

constexpr int TILE = 128;
constexpr int UNIT = 64;
constexpr int NTHREADS = 576;
constexpr int WARP_TMA = 16, WARP_MMA = 17;
constexpr int COLS = 32;  // columns of a compute warp
constexpr int kCtas = 148;  // one per SM
constexpr float kLog2e = 1.4426950408889634f;
constexpr int HALF = TILE * 128;   // 64 columns of a 128-row tile: rows of 128 bytes
constexpr int UHALF = UNIT * 128;  // 64 columns of a unit's rows
constexpr int ROWB = UNIT * 4;     // one fp32 row vector of a unit

template <int HD>
struct Cfg {
  static constexpr int TB = TILE * HD * 2, UB = UNIT * HD * 2;  // a tile, a unit
  static constexpr uint32_t IDESC_U = idesc_bf16_f32(TILE, UNIT, false, false);
  static constexpr uint32_t IDESC_T = idesc_bf16_f32(TILE, TILE, false, false);
  static constexpr uint32_t IDESC_ACC = idesc_bf16_f32(TILE, HD, false, true);
};

struct BwdParams {
  TensorRef q, k, v, up, dq, dk, dv;  // up: the upstream gradient
  const float* lse2;
  const float* dsum;
  float* part;
  int32_t* status;
  int B, Hq, Hkv, g, N, Npad, NT, window, sinks, L, partials, cut;
  int zq, zk, zv, zg;  // broadcast dimensions: bit 0 batch, bit 1 head
  float c, scale;      // c = scale * log2(e)
  bool wide_q, wide_kv;  // gradients in 32-byte pieces
};

// D (128 x R) = A B^T over HD: a 128-row tile and R rows (a tile's or a unit's), both K-major in shared memory
// (low descriptor words).
template <int HD, int R>
__device__ __forceinline__ void mma_logits(uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk)
    mma_ss_lo(d, a + (((kk >> 2) * HALF + (kk & 3) * 32) >> 4), b + (((kk >> 2) * R * 128 + (kk & 3) * 32) >> 4),
              R == UNIT ? Cfg<HD>::IDESC_U : Cfg<HD>::IDESC_T, kk > 0 ? 1u : 0u);
}
__device__ __forceinline__ uint32_t kmajor(uint32_t saddr) { return desc_lo(saddr, 16); }
__device__ __forceinline__ uint32_t mnmajor(uint32_t saddr, uint32_t half) { return desc_lo(saddr, half); }

// D (128 x HD) (+)= A B, A 128 x R as bf16 pairs in TMEM (32 of the reduction in columns a + 32 i .. + 15),
// B the R rows (the reduction) of a tile or a unit in shared memory (low descriptor word).
template <int HD, int R>
__device__ __forceinline__ void mma_grad(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
#pragma unroll
  for (int kk = 0; kk < R / 16; ++kk)
    mma_ts_lo(d, a + 32 * (kk >> 1) + 8 * (kk & 1), b + kk * 128, Cfg<HD>::IDESC_ACC, kk > 0 ? 1u : acc);
}

// Rows of a tile or a unit (`half`: bytes of 64 of its columns).
template <int HD>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int row, int h, int b,
                                          int zero, int half) {
#pragma unroll
  for (int f = 0; f < HD / 64; ++f)
    tma_load_4d(dst + f * half, map, bar, 64 * f, row, zero & 2 ? 0 : h, zero & 1 ? 0 : b);
}

// Shared memory is filled to the last kilobyte: its start has to be a 1024-byte boundary as it is.
__device__ __forceinline__ bool misaligned(const uint8_t* smem, int32_t* status) {
  if ((smem_u32(smem) & 1023u) == 0) return false;
  if (threadIdx.x == 0) atomicCAS(status, 0, (int)SSA_ERR_CUDA);
  return true;
}

// 16 columns of an accumulator row, scaled, to bf16 memory.
__device__ __forceinline__ void store16(bf16* dst, const uint32_t (&r)[16], float mul, bool wide) {
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = pack_bf16(__uint_as_float(r[2 * i]) * mul, __uint_as_float(r[2 * i + 1]) * mul);
  store_32b(dst, o, wide);
}

// z becomes NaN where one of 16 values is not finite.
__device__ __forceinline__ void look16(float2& z, const uint32_t (&r)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 2)
    z = fma2(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), make_float2(0.f, 0.f), z);
}

// ================================================================ dK, dV
template <int HD>
struct DkvCfg {
  static constexpr int NS = HD == 128 ? 5 : 8;  // units in flight
  static constexpr int TB = Cfg<HD>::TB, UB = Cfg<HD>::UB;
  static constexpr int OFF_V = TB, OFF_Q = 2 * TB, OFF_ROW = OFF_Q + NS * 2 * UB;  // Q, g of each unit; -lse2, -D
  static constexpr int OFF_MISC = OFF_ROW + NS * 2 * ROWB;
};
struct DkvMisc {
  uint64_t kv_full, q_full[8], q_empty[8], s_full[2], p_full[2], dp_full[2], ds_full[2], done, drain;
  uint32_t tmem_base;
  int abort;
};

template <int HD>
__global__ void __launch_bounds__(NTHREADS, 1)
    win_bwd_dkv_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
                          const __grid_constant__ BwdParams p) {
  using C = DkvCfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (misaligned(smem, p.status)) return;
  DkvMisc& M = *reinterpret_cast<DkvMisc*>(smem + C::OFF_MISC);
  volatile int* abort = &M.abort;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
  const int plane = (int)blockIdx.x % p.Hkv + (int)blockIdx.y * p.Hkv, kvh = plane % p.Hkv, b = blockIdx.y;

  if (threadIdx.x == 0) {
    mbar_init(&M.kv_full, 1);
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&M.q_full[i], 1);
      mbar_init(&M.q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&M.s_full[i], 1);
      mbar_init(&M.p_full[i], 8);
      mbar_init(&M.dp_full[i], 1);
      mbar_init(&M.ds_full[i], 8);
    }
    mbar_init(&M.done, 1);
    mbar_init(&M.drain, 1);
    M.abort = 0;
    fence_mbar_init();
  }
  if (warp == WARP_MMA) {
    tmem_alloc(&M.tmem_base, 512);
    tmem_relinquish();
  }
  const Chunk ch = find_chunk<TILE>((int)blockIdx.x / p.Hkv, p.cut, p.L, p.g, p.N, p.window, p.sinks);
  const int u0 = ch.kt * TILE, nq = query_tiles_of<TILE>(ch.kt, p.N, p.window, p.sinks);
  const int first = ch.idx * p.L, T = 2 * min(p.L, nq * p.g - first);  // units: step (head, query tile), half
  bool again = false;  // the thread's row is not finite
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  allow_ahead();
  ahead_wait();
  const uint32_t tmem = M.tmem_base;
  const uint32_t cK = tmem, cV = tmem + HD, cS = tmem + 256, cP = tmem + 384;
  uint8_t* sK = smem;
  uint8_t* sV = smem + C::OFF_V;
  auto unit = [&](int i) { return smem + C::OFF_Q + (i % C::NS) * 2 * C::UB; };
  auto rows = [&](int i) { return smem + C::OFF_ROW + (i % C::NS) * 2 * ROWB; };

  if (warp == WARP_TMA) {
    if (elect_one()) {
      prefetch_tensormap(&tmQ);
      prefetch_tensormap(&tmG);
      mbar_expect_tx(&M.kv_full, 2 * C::TB);
      load_tile<HD>(sK, &tmK, &M.kv_full, u0, kvh, b, p.zk, HALF);
      load_tile<HD>(sV, &tmV, &M.kv_full, u0, kvh, b, p.zv, HALF);
      int issued = 0, h = kvh * p.g + first / nq, qt = first % nq;
      for (int i = 0; i < T; ++i) {
        uint64_t* full = &M.q_full[i % C::NS];
        if (i >= C::NS && !mbar_wait(&M.q_empty[i % C::NS], (uint32_t)(i / C::NS - 1) & 1u, abort)) break;
        const int t0 = (ch.kt + qt) * TILE + (i & 1) * UNIT;
        const int64_t ro = ((int64_t)b * p.Hq + h) * p.Npad + t0;
        mbar_expect_tx(full, 2 * C::UB + 2 * ROWB);
        load_tile<HD>(unit(i), &tmQ, full, t0, h, b, p.zq, UHALF);
        bulk_load(rows(i), p.lse2 + ro, ROWB, full);
        load_tile<HD>(unit(i) + C::UB, &tmG, full, t0, h, b, p.zg, UHALF);
        bulk_load(rows(i) + ROWB, p.dsum + ro, ROWB, full);
        issued = i + 1;
        if (i & 1)
          if (++qt == nq) {
            qt = 0;
            ++h;
          }
      }
      int dummy = 0;
      mbar_wait(&M.kv_full, 0, &dummy);
      for (int i = issued > C::NS ? issued - C::NS : 0; i < issued; ++i) {
        dummy = 0;
        mbar_wait(&M.q_full[i % C::NS], (uint32_t)(i / C::NS) & 1u, &dummy);
      }
    }
    __syncwarp();
  } else if (warp == WARP_MMA) {
    if (elect_one()) {
      const uint32_t ak = kmajor(smem_u32(sK)), av = kmajor(smem_u32(sV));
      const uint32_t bq = kmajor(smem_u32(smem + C::OFF_Q)), mq = mnmajor(smem_u32(smem + C::OFF_Q), UHALF);
      constexpr uint32_t US = 2 * C::UB >> 4, G = C::UB >> 4;  // from unit to unit, from Q to g
      auto slot = [&](int i) { return (uint32_t)(i % C::NS) * US; };
      auto have = [&](int i) { return mbar_wait(&M.q_full[i % C::NS], (uint32_t)(i / C::NS) & 1u, abort); };
      auto s_of = [&](int i) {
        mma_logits<HD, UNIT>(cS + UNIT * (i & 1), ak, bq + slot(i));
        tc_commit(&M.s_full[i & 1]);
      };
      auto dp_of = [&](int i) {
        mma_logits<HD, UNIT>(cP + UNIT * (i & 1), av, bq + slot(i) + G);
        tc_commit(&M.dp_full[i & 1]);
      };
      bool ok = mbar_wait(&M.kv_full, 0, abort) && have(0);
      if (ok) {
        tc_fence_after();
        s_of(0);
        dp_of(0);
        if ((ok = have(1))) {  // T is even
          tc_fence_after();
          s_of(1);
        }
      }
      for (int i = 0; ok && i <= T; ++i) {
        if (i < T) {
          if (!(ok = mbar_wait(&M.p_full[i & 1], (uint32_t)(i >> 1) & 1u, abort))) break;
          tc_fence_after();
          mma_grad<HD, UNIT>(cV, cS + UNIT * (i & 1), mq + slot(i) + G, i > 0 ? 1u : 0u);
          if (i + 2 < T) {
            if (!(ok = have(i + 2))) break;
            tc_fence_after();
            s_of(i + 2);
          }
        }
        if (i > 0) {
          const int k = i - 1;
          if (!(ok = mbar_wait(&M.ds_full[k & 1], (uint32_t)(k >> 1) & 1u, abort))) break;
          tc_fence_after();
          mma_grad<HD, UNIT>(cK, cP + UNIT * (k & 1), mq + slot(k), k > 0 ? 1u : 0u);
          tc_commit(&M.q_empty[k % C::NS]);
        }
        if (i + 1 < T) dp_of(i + 1);
      }
      tc_commit(&M.done);
      tc_commit(&M.drain);
      int dummy = 0;
      mbar_wait(&M.drain, 0, &dummy);
    }
    __syncwarp();
  } else {
    // key rows 32 quarter.., query columns 32 cg.. of the group's units
    const int quarter = warp & 3, cg = (warp >> 2) & 1, grp = warp >> 3;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t aS = cS + lane_base + UNIT * grp + COLS * cg, aP = cP + lane_base + UNIT * grp + COLS * cg;
    const int u = u0 + quarter * 32 + lane;
    const int ua = u0 + quarter * 32, ub = ua + 31;
    const float2 cc = make_float2(p.c, p.c);
    int qt = first % nq;  // query tile of the step, from the key tile on
    bool ok = true;
    for (int i = grp; i < T; i += 2) {
      const uint32_t ph = (uint32_t)(i >> 1);
      const int t0 = (ch.kt + qt) * TILE + UNIT * grp + COLS * cg;  // this warp's first query
      if (++qt == nq) qt = 0;
      const float* ls = reinterpret_cast<const float*>(rows(i)) + COLS * cg;
      const float* ds = ls + UNIT;
      // every lane reads the unit's row vectors: every lane waits for them
      if (!__all_sync(0xffffffffu, mbar_wait(&M.q_full[i % C::NS], (uint32_t)(i / C::NS) & 1u, abort)) ||
          !__all_sync(0xffffffffu, mbar_wait(&M.s_full[grp], ph & 1u, abort))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool all = t0 >= ub && (t0 + COLS - 1 - ua < p.window || ub < p.sinks);
      const uint32_t vis = visible_queries(u, t0, p.window, p.sinks);
      float x[COLS];
      tmem_ld32(aS, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
      tmem_wait_ld();
      uint32_t pk[COLS / 2];
#pragma unroll
      for (int c = 0; c < COLS; c += 4) {
        const float4 l4 = *reinterpret_cast<const float4*>(ls + c);  // -lse2
        const float2 y0 = fma2(make_float2(x[c], x[c + 1]), cc, make_float2(l4.x, l4.y));
        const float2 y1 = fma2(make_float2(x[c + 2], x[c + 3]), cc, make_float2(l4.z, l4.w));
        x[c] = ex2(y0.x);
        x[c + 1] = ex2(y0.y);
        x[c + 2] = ex2(y1.x);
        x[c + 3] = ex2(y1.y);
      }
      if (!all) {
#pragma unroll
        for (int c = 0; c < COLS; ++c) x[c] = keep(vis, c, x[c], 0.f);
      }
#pragma unroll
      for (int c = 0; c < COLS; c += 2) pk[c / 2] = pack_bf16(x[c], x[c + 1]);
      tmem_st16(aS, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&M.p_full[grp]);

      if (!__all_sync(0xffffffffu, mbar_wait(&M.dp_full[grp], ph & 1u, abort))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t y[COLS];
      tmem_ld32(aP, y);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < COLS; c += 4) {
        const float4 d4 = *reinterpret_cast<const float4*>(ds + c);  // -D
        const float2 z0 = mul2(make_float2(x[c], x[c + 1]),
                               add2(make_float2(__uint_as_float(y[c]), __uint_as_float(y[c + 1])), make_float2(d4.x, d4.y)));
        const float2 z1 = mul2(make_float2(x[c + 2], x[c + 3]),
                               add2(make_float2(__uint_as_float(y[c + 2]), __uint_as_float(y[c + 3])), make_float2(d4.z, d4.w)));
        x[c] = z0.x;
        x[c + 1] = z0.y;
        x[c + 2] = z1.x;
        x[c + 3] = z1.y;
      }
      if (!all) {  // zero times a NaN or an infinity of a hidden pair
#pragma unroll
        for (int c = 0; c < COLS; ++c) x[c] = keep(vis, c, x[c], 0.f);
      }
#pragma unroll
      for (int c = 0; c < COLS; c += 2) pk[c / 2] = pack_bf16(x[c], x[c + 1]);
      tmem_st16(aP, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&M.ds_full[grp]);
    }
    if (ok && __all_sync(0xffffffffu, mbar_wait(&M.done, 0, abort))) {
      tc_fence_after();
      // columns HD/4 (warp / 4) .. of dK and dV
      constexpr int W = HD / 4;
      const int col0 = W * (warp >> 2);
      const bool mine = u < p.N;
      float* part = p.part + ((size_t)plane * p.partials + ch.slot + ch.idx) * (2 * TILE * HD) +
                    (quarter * 32 + lane) * HD + col0;
      float2 z = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int c0 = 0; c0 < 2 * W; c0 += 16) {
        const int which = c0 / W, col = c0 % W;  // 0: dK, 1: dV
        uint32_t r[16];
        tmem_ld16((which ? cV : cK) + lane_base + col0 + col, r);
        tmem_wait_ld();
        if (!mine) continue;
        look16(z, r);
        if (ch.n == 1) {
          const TensorRef& t = which ? p.dv : p.dk;
          store16(row_ptr_w<bf16>(t, b, kvh, u) + col0 + col, r, which ? 1.0f : p.scale, p.wide_kv);
        } else {
          uint4* d4 = reinterpret_cast<uint4*>(part + which * TILE * HD + col);
#pragma unroll
          for (int v = 0; v < 4; ++v) d4[v] = make_uint4(r[4 * v], r[4 * v + 1], r[4 * v + 2], r[4 * v + 3]);
        }
      }
      again = z.x + z.y != 0.f;
    }
  }
  tc_fence_before();
  const bool spoilt = __syncthreads_or(again) && !M.abort;
  if (M.abort && threadIdx.x == 0) atomicCAS(p.status, 0, (int)SSA_ERR_TIMEOUT);
  if (warp == WARP_MMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // rows that are not finite once more (win_rows.cuh)
  if (!spoilt) return;
  const QueryView view{p.q, p.up, p.lse2, p.dsum, b, p.Hq, kvh * p.g, ch.kt, nq, first, first + T / 2, p.N, p.Npad, p.window, p.sinks};
  for (int r = warp; r < TILE && u0 + r < p.N; r += NTHREADS / 32) {
    const int u = u0 + r;
    float* part = ch.n == 1 ? nullptr : p.part + ((size_t)plane * p.partials + ch.slot + ch.idx) * (2 * TILE * HD) + r * HD;
    mend_dkv_row<bf16, HD, TILE>(view, u, row_ptr<bf16>(p.k, b, kvh, u), row_ptr<bf16>(p.v, b, kvh, u), row_ptr_w<bf16>(p.dk, b, kvh, u),
                                 row_ptr_w<bf16>(p.dv, b, kvh, u), part, part == nullptr ? nullptr : part + TILE * HD, p.c, p.scale);
  }
}

// ================================================================ dQ
template <int HD>
struct DqCfg {
  static constexpr int NSK = HD == 128 ? 3 : 5, NSV = HD == 128 ? 2 : 4;  // K, V tiles in flight
  static constexpr int TB = Cfg<HD>::TB;
  static constexpr int OFF_G = TB, OFF_K = 2 * TB, OFF_V = OFF_K + NSK * TB, OFF_MISC = OFF_V + NSV * TB;
};
struct DqMisc {
  uint64_t q_full, q_empty, k_full[5], k_empty[5], v_full[4], v_empty[4];
  uint64_t s_full[2], dp_full, ds_full, dq_done, dq_free, drain;
  uint32_t tmem_base;
  int abort;
};

struct DqItem {
  int b, h, kvh, t0;
  KeyTiles kt;
};

template <int HD>
__global__ void __launch_bounds__(NTHREADS, 1)
    win_bwd_dq_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
                         const __grid_constant__ CUtensorMap tmKs, const __grid_constant__ BwdParams p) {
  using C = DqCfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (misaligned(smem, p.status)) return;
  DqMisc& M = *reinterpret_cast<DqMisc*>(smem + C::OFF_MISC);
  volatile int* abort = &M.abort;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform

  if (threadIdx.x == 0) {
    mbar_init(&M.q_full, 1);
    mbar_init(&M.q_empty, 1);
    for (int i = 0; i < C::NSK; ++i) {
      mbar_init(&M.k_full[i], 1);
      mbar_init(&M.k_empty[i], 1);
    }
    for (int i = 0; i < C::NSV; ++i) {
      mbar_init(&M.v_full[i], 1);
      mbar_init(&M.v_empty[i], 1);
    }
    mbar_init(&M.s_full[0], 1);
    mbar_init(&M.s_full[1], 1);
    mbar_init(&M.dp_full, 1);
    mbar_init(&M.ds_full, 16);
    mbar_init(&M.dq_done, 1);
    mbar_init(&M.dq_free, 16);
    mbar_init(&M.drain, 1);
    M.abort = 0;
    fence_mbar_init();
  }
  if (warp == WARP_MMA) {
    tmem_alloc(&M.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  ahead_wait();
  const uint32_t tmem = M.tmem_base;
  const uint32_t cQ = tmem, cS = tmem + 128, cP = tmem + 384;
  uint8_t* sQ = smem;
  uint8_t* sG = smem + C::OFF_G;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;

  bool again = false;  // the thread stored rows that are not finite
  const int planes = p.B * p.Hq, items = planes * p.NT;
  // The longest rows first; the heads of a group side by side, so that they share K and V in L2.
  auto item = [&](int i) {
    DqItem I;
    const int plane = i % planes;
    I.t0 = (p.NT - 1 - i / planes) * TILE;
    I.b = plane / p.Hq;
    I.h = plane % p.Hq;
    I.kvh = I.h / p.g;
    I.kt = key_tiles<TILE>(I.t0, min(I.t0 + TILE, p.N) - 1, p.window, p.sinks);
    return I;
  };

  if (warp == WARP_TMA) {
    if (elect_one()) {
      prefetch_tensormap(&tmQ);
      prefetch_tensormap(&tmK);
      prefetch_tensormap(&tmV);
      prefetch_tensormap(&tmG);
      uint32_t n = 0, qn = 0, kn = 0, vn = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
        const DqItem I = item(i);
        if (qn > 0 && !mbar_wait(&M.q_empty, (qn - 1) & 1u, abort)) break;
        mbar_expect_tx(&M.q_full, 2 * C::TB);
        load_tile<HD>(sQ, &tmQ, &M.q_full, I.t0, I.h, I.b, p.zq, HALF);
        load_tile<HD>(sG, &tmG, &M.q_full, I.t0, I.h, I.b, p.zg, HALF);
        ++qn;
        for (int j = 0; j < I.kt.count; ++j, ++n) {
          const int u0 = I.kt.tile(j) * TILE, ik = (int)(n % C::NSK), iv = (int)(n % C::NSV);
          if (n >= C::NSK && !(ok = mbar_wait(&M.k_empty[ik], (n / C::NSK - 1) & 1u, abort))) break;
          mbar_expect_tx(&M.k_full[ik], C::TB);
          // a sink tile's K through a map that ends at the sinks: no query of the item sees its other keys
          load_tile<HD>(sK + ik * C::TB, j < I.kt.ns ? &tmKs : &tmK, &M.k_full[ik], u0, I.kvh, I.b, p.zk, HALF);
          kn = n + 1;
          if (n >= C::NSV && !(ok = mbar_wait(&M.v_empty[iv], (n / C::NSV - 1) & 1u, abort))) break;
          mbar_expect_tx(&M.v_full[iv], C::TB);
          load_tile<HD>(sV + iv * C::TB, &tmV, &M.v_full[iv], u0, I.kvh, I.b, p.zv, HALF);
          vn = n + 1;
        }
      }
      int dummy = 0;
      if (qn) mbar_wait(&M.q_full, (qn - 1) & 1u, &dummy);
      for (uint32_t k = kn > C::NSK ? kn - C::NSK : 0; k < kn; ++k) {
        dummy = 0;
        mbar_wait(&M.k_full[k % C::NSK], (k / C::NSK) & 1u, &dummy);
      }
      for (uint32_t k = vn > C::NSV ? vn - C::NSV : 0; k < vn; ++k) {
        dummy = 0;
        mbar_wait(&M.v_full[k % C::NSV], (k / C::NSV) & 1u, &dummy);
      }
    }
    __syncwarp();
  } else if (warp == WARP_MMA) {
    if (elect_one()) {
      const uint32_t aq = kmajor(smem_u32(sQ)), ag = kmajor(smem_u32(sG)), bk = kmajor(smem_u32(sK)), bv = kmajor(smem_u32(sV));
      const uint32_t mk = mnmajor(smem_u32(sK), HALF);
      constexpr uint32_t TS = C::TB >> 4;
      uint32_t n = 0, qn = 0;  // tiles and items so far
      bool ok = true;
      auto s_of = [&](uint32_t k) {
        if (!mbar_wait(&M.k_full[k % C::NSK], (k / C::NSK) & 1u, abort)) return false;
        tc_fence_after();
        mma_logits<HD, TILE>(cS + TILE * (k & 1), aq, bk + (k % C::NSK) * TS);
        tc_commit(&M.s_full[k & 1]);
        return true;
      };
      auto dp_of = [&](uint32_t k) {
        if (!mbar_wait(&M.v_full[k % C::NSV], (k / C::NSV) & 1u, abort)) return false;
        tc_fence_after();
        mma_logits<HD, TILE>(cP, ag, bv + (k % C::NSV) * TS);
        tc_commit(&M.dp_full);
        tc_commit(&M.v_empty[k % C::NSV]);
        return true;
      };
      for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
        const int T = item(i).kt.count;
        if (!(ok = mbar_wait(&M.q_full, qn & 1u, abort))) break;
        tc_fence_after();
        ok = s_of(n) && dp_of(n) && (T < 2 || s_of(n + 1));
        if (T == 1) tc_commit(&M.q_empty);
        // every warp has read the item before's dQ
        if (ok && qn > 0) ok = mbar_wait(&M.dq_free, (qn - 1) & 1u, abort);
        ++qn;
        for (int j = 0; ok && j < T; ++j, ++n) {
          if (!(ok = mbar_wait(&M.ds_full, n & 1u, abort))) break;  // dP(j) is read, dx(j) written
          tc_fence_after();
          if (j + 1 < T && !(ok = dp_of(n + 1))) break;
          if (j + 2 == T) tc_commit(&M.q_empty);  // the last S and dP of the item are issued
          mma_grad<HD, TILE>(cQ, cS + TILE * (n & 1), mk + (n % C::NSK) * TS, j > 0 ? 1u : 0u);
          tc_commit(&M.k_empty[n % C::NSK]);
          if (j + 1 == T) tc_commit(&M.dq_done);
          if (j + 2 < T) ok = s_of(n + 2);
        }
      }
      tc_commit(&M.drain);
      int dummy = 0;
      mbar_wait(&M.drain, 0, &dummy);
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3, cg = warp >> 2;  // query rows 32 quarter.., key columns 32 cg..
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t aP = cP + lane_base + COLS * cg;
    uint32_t n = 0, qn = 0;
    bool ok = true;
    float2 z = make_float2(0.f, 0.f);  // NaN behind a row that is not finite
    DqItem I = item(blockIdx.x);
    float nl, nd;  // -lse2, -D
    auto statistics = [&](const DqItem& J) {
      const int64_t ro = ((int64_t)J.b * p.Hq + J.h) * p.Npad + J.t0 + quarter * 32 + lane;
      nl = p.lse2[ro];
      nd = p.dsum[ro];
    };
    statistics(I);
    for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
      const int t = I.t0 + quarter * 32 + lane, ta = I.t0 + quarter * 32, tb = ta + 31;
      const float2 cc = make_float2(p.c, p.c), ll = make_float2(nl, nl), dd = make_float2(nd, nd);
      for (uint32_t k = n; k < n + I.kt.count; ++k) {
        if (!__all_sync(0xffffffffu, mbar_wait(&M.s_full[k & 1], (k >> 1) & 1u, abort))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t aS = cS + lane_base + TILE * (k & 1) + COLS * cg;
        const int u0 = I.kt.tile((int)(k - n)) * TILE + COLS * cg;  // this warp's first key
        const bool all = u0 + COLS - 1 <= ta && (tb - u0 < p.window || u0 + COLS <= p.sinks);
        float x[COLS];
        tmem_ld32(aS, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < COLS; c += 2) {
          const float2 y = fma2(make_float2(x[c], x[c + 1]), cc, ll);
          x[c] = ex2(y.x);
          x[c + 1] = ex2(y.y);
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&M.dp_full, k & 1u, abort))) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t y[COLS], pk[COLS / 2];
        tmem_ld32(aP, y);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < COLS; c += 2) {
          const float2 z = mul2(make_float2(x[c], x[c + 1]), add2(make_float2(__uint_as_float(y[c]), __uint_as_float(y[c + 1])), dd));
          x[c] = z.x;
          x[c + 1] = z.y;
        }
        if (!all) {
          const uint32_t vis = visible_keys(t, u0, p.window, p.sinks);
#pragma unroll
          for (int c = 0; c < COLS; ++c) x[c] = keep(vis, c, x[c], 0.f);
        }
#pragma unroll
        for (int c = 0; c < COLS; c += 2) pk[c / 2] = pack_bf16(x[c], x[c + 1]);
        tmem_st16(aS, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M.ds_full);
      }
      n += I.kt.count;
      // The next item's coordinates and statistics are fetched while the last product runs.
      DqItem J = I;
      if (i + (int)gridDim.x < items) {
        J = item(i + gridDim.x);
        statistics(J);
      }
      if (!ok || !__all_sync(0xffffffffu, mbar_wait(&M.dq_done, qn & 1u, abort))) break;
      ++qn;
      tc_fence_after();
      constexpr int W = HD / 4;
#pragma unroll 1
      for (int c0 = 0; c0 < W; c0 += 16) {
        uint32_t r[16];
        tmem_ld16(cQ + lane_base + W * cg + c0, r);
        tmem_wait_ld();
        if (t < p.N) {
          look16(z, r);
          store16(row_ptr_w<bf16>(p.dq, I.b, I.h, t) + W * cg + c0, r, p.scale, p.wide_q);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&M.dq_free);
      I = J;
    }
    again = z.x + z.y != 0.f;
  }
  tc_fence_before();
  const bool spoilt = __syncthreads_or(again) && !M.abort;
  if (M.abort && threadIdx.x == 0) atomicCAS(p.status, 0, (int)SSA_ERR_TIMEOUT);
  if (warp == WARP_MMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // they are formed once more (win_rows.cuh)
  for (int i = blockIdx.x; spoilt && i < items; i += gridDim.x) {
    const DqItem I = item(i);
    const KeyRows<bf16> keys{p.k, p.v, I.b, I.kvh, nullptr, 0, 0, 0};
    for (int t = I.t0 + warp; t < min(I.t0 + TILE, p.N); t += NTHREADS / 32) {
      const int64_t o = ((int64_t)I.b * p.Hq + I.h) * p.Npad + t;
      const RowView view{I.kt, t, 0, I.kt.count, p.window, p.sinks, p.N};
      mend_dq_row<bf16, HD, TILE>(keys, view, row_ptr<bf16>(p.q, I.b, I.h, t), row_ptr<bf16>(p.up, I.b, I.h, t),
                                  row_ptr_w<bf16>(p.dq, I.b, I.h, t), p.c, p.lse2[o], p.dsum[o], p.scale);
    }
  }
}

template <int HD>
constexpr int dkv_smem() {
  return DkvCfg<HD>::OFF_MISC + (int)sizeof(DkvMisc);
}
template <int HD>
constexpr int dq_smem() {
  return DqCfg<HD>::OFF_MISC + (int)sizeof(DqMisc);
}
static_assert(dkv_smem<128>() <= 232448 && dq_smem<128>() <= 232448, "shared memory of a CTA");

template <int HD>
cudaError_t launch(const WinDims& D, const WinBwdArgs& a, int32_t* status, cudaStream_t st) {
  BwdParams p{};
  // Boxes of 128 rows, and of 64 for the units of queries.
  CUtensorMap q, k, ks, v, g, qu, gu;
  auto map = [&](CUtensorMap* m, const TensorRef& t, int H, int rows, int* zero) {
    return win_tma_map(m, t, D.B, H, D.N, rows, HD, zero);
  };
  if (!win_tma_map(&ks, a.k, D.B, D.Hkv, D.sinks > 0 ? D.sinks : D.N, TILE, HD, &p.zk)) return cudaErrorInvalidValue;
  if (!map(&q, a.q, D.Hq, TILE, &p.zq) || !map(&g, a.g, D.Hq, TILE, &p.zg) || !map(&k, a.k, D.Hkv, TILE, &p.zk) ||
      !map(&v, a.v, D.Hkv, TILE, &p.zv) || !map(&qu, a.q, D.Hq, UNIT, &p.zq) || !map(&gu, a.g, D.Hq, UNIT, &p.zg))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_win_bwd_pre(D, a, st);
  if (e != cudaSuccess) return e;
  const WinBwdLayout L = win_bwd_layout(D);
  const ChunkPlan cp = chunk_plan<TILE>(D, kBwdChunks, kTcMinSteps);
  char* ws = static_cast<char*>(a.ws);
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.up = a.g;
  p.dq = a.dq;
  p.dk = a.dk;
  p.dv = a.dv;
  p.lse2 = reinterpret_cast<const float*>(ws + L.lse2);
  p.dsum = reinterpret_cast<const float*>(ws + L.dsum);
  p.part = reinterpret_cast<float*>(ws + L.part);
  p.status = status;
  p.B = D.B;
  p.Hq = D.Hq;
  p.Hkv = D.Hkv;
  p.g = D.g;
  p.N = D.N;
  p.Npad = L.Npad;
  p.NT = cp.NT;
  p.window = D.window;
  p.sinks = D.sinks;
  p.L = cp.L;
  p.partials = cp.partials;
  p.cut = cp.cut;
  p.c = D.scale * kLog2e;
  p.scale = D.scale;
  p.wide_q = wide_rows(a.dq);
  p.wide_kv = wide_rows(a.dk) && wide_rows(a.dv);
  auto dkv = win_bwd_dkv_tc_kernel<HD>;
  if ((e = cudaFuncSetAttribute(dkv, cudaFuncAttributeMaxDynamicSharedMemorySize, dkv_smem<HD>())) != cudaSuccess) return e;
  if ((e = launch_ahead(dkv, dim3(cp.chunks * D.Hkv, D.B), NTHREADS, dkv_smem<HD>(), st, qu, k, v, gu, p)) != cudaSuccess) return e;
  if ((e = launch_win_kvjoin<TILE>(D, a, cp, p.part, st)) != cudaSuccess) return e;
  auto dq = win_bwd_dq_tc_kernel<HD>;
  if ((e = cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, dq_smem<HD>())) != cudaSuccess) return e;
  const int64_t items = (int64_t)D.B * D.Hq * cp.NT;
  return launch_ahead(dq, dim3((unsigned)(items < kCtas ? items : kCtas)), NTHREADS, dq_smem<HD>(), st, q, k, v, g, ks, p);
}

}  // namespace

cudaError_t launch_win_bwd_tc(const WinDims& D, const WinBwdArgs& a, int32_t* status, cudaStream_t st) {
  return D.d == 64 ? launch<64>(D, a, status, st) : launch<128>(D, a, status, st);
}

}  // namespace ssa
