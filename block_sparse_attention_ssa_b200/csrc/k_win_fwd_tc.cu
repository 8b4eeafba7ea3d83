// Window attention with sinks and paged attention on tcgen05 (bf16, d = 64 or 128).
//
// Mathematics: for each query the online softmax over its visible keys in base 2 with
// the scale folded in, p = 2^(s c - m), c = scale log2(e); the running maximum m is
// raised only when a tile exceeds it by more than 8 (p stays below 2^8), so the
// accumulator is rarely rescaled.  Logits, statistics and sums are fp32; p is rounded to
// bf16 as an operand of the second product (half a step, 2^-8 of a weight, averaged over
// the row), its sum is taken before the rounding.
//
// A persistent CTA per SM walks work items of up to 256 query rows in two slots of 128
// (TMEM lanes): warps 0-3 hold slot 0's softmax, warps 4-7 slot 1's, warp 8 loads by TMA,
// warp 9 issues the products.  While one slot's softmax works, the tensor core runs the
// other slot's products; the key tiles (128 keys) are shared by both.  TMEM: O of slot s
// at HD s, S of slot s at 256 + 128 s; P (bf16 pairs) overwrites the second half of S and
// feeds P V from TMEM.  An item whose rows fit one slot gives the odd key tiles to slot 1
// with the same queries, and slot 0's warps join the two softmaxes at the end, so that a
// decoding step has two chains in flight too.
//
// Rows.  Window form: a row is a token of one query head.  Paged form: a row is a
// (new token, head of the group) pair, so the g heads of a kv head share each K/V load
// and a single token fills g rows; 128 / g tokens to a slot.  Paged items are cut into
// equal shares of key tiles (win_common.cuh); cut items leave fp32 partials.
#include "win_common.cuh"

#include "sm100_ptx.cuh"

namespace ssa {
namespace {

using namespace sm100;
using bf16 = __nv_bfloat16;

constexpr int TILE = 128;
constexpr int NTHREADS = 320;
constexpr int WARP_TMA = 8, WARP_MMA = 9;
constexpr int kCtas = 148;     // one per SM
constexpr int kMinUnits = 4;   // key tiles worth a CTA of their own
constexpr float kRescaleThreshold = 8.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t COL_S = 256;

template <int HD>
struct Cfg {
  static constexpr int NSK = HD == 128 ? 3 : 4, NSV = HD == 128 ? 2 : 4;  // K, V tiles in flight
  static constexpr int TB = TILE * HD * 2;
  static constexpr int HALF = TILE * 128;  // 64 columns of a tile: 128 rows of 128 bytes
  static constexpr int OFF_K = 2 * TB, OFF_V = OFF_K + NSK * TB, OFF_MISC = OFF_V + NSV * TB;
  static constexpr uint32_t IDESC_S = idesc_bf16_f32(TILE, TILE, false, false);
  static constexpr uint32_t IDESC_PV = idesc_bf16_f32(TILE, HD, false, true);
};

struct Misc {
  uint64_t q_full, q_empty, k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], p_full[2], pv_done[2], join_ready, join_done, drain;
  uint32_t tmem_base;
  int abort;
  int left;
  Place at;
  uint32_t bad[8];  // pages missing from a key tile, a bit per 16 keys (ring of 2 NSK tiles)
  float jm[TILE], jl[TILE];
};

struct TcParams {
  TensorRef h;
  float* lse;
  int32_t* status;
  int B, Hq, g, N, window, sinks;
  int zk, zv, zq;    // broadcast dimensions of K, V, Q: bit 0 batch, bit 1 head
  int rows_item;     // window form: tokens of an item (256, or 128 when those would leave SMs idle)
  float c;           // scale * log2(e)
  // paged form
  const int32_t* table;
  Batch batch;
  int page, num_pages, max_pages, TQ;
  float* part;
};

// One work item as its roles see it.
struct Item {
  int b, kvh, head0, row0, p0, g;   // row0: first token (window) or packed row (paged); p0: its position
  int toks0, toks1;                 // tokens of the two slots
  int T, off, seg, units;           // key tiles of this CTA's share, the first one's index
  bool two, cut;                    // both slots hold rows; share of an item only
  KeyTiles kt;
  int ns0, lo0, hi0, ns1, lo1, hi1; // two: the tiles that each slot sees
  int step;                         // tokens of a full slot
  __device__ __forceinline__ int tile(int j) const { return kt.tile(off + j); }
  __device__ __forceinline__ bool active(int s, int j) const {
    if (!two) return (j & 1) == s;
    const int t = tile(j);
    return t < (s ? ns1 : ns0) || (t >= (s ? lo1 : lo0) && t <= (s ? hi1 : hi0));
  }
  __device__ __forceinline__ int next(int s, int j) const {
    while (j < T && !active(s, j)) ++j;
    return j;
  }
};

template <bool PAGED>
struct Walk {
  const TcParams& p;
  Place at;
  int left, idx, seg;
  __device__ Walk(const TcParams& p_, const Misc& M) : p(p_), at(M.at), left(M.left), idx(blockIdx.x), seg(0) {}

  __device__ bool next(Item& I) {
    int toks, cap;
    if (PAGED) {
      if (left <= 0 || at.b >= p.batch.seqs) return false;
      const Seq s = load_seq(p.batch.q_start, p.batch.kv_len, at.b, p.batch.T, p.batch.cap);
      const int i0 = at.run * p.batch.TI;
      toks = min(p.batch.TI, s.n - i0);
      cap = p.TQ;
      I.b = at.b;
      I.kvh = at.kvh;
      I.head0 = at.kvh * p.g;
      I.g = p.g;
      I.row0 = s.q0 + i0;
      I.p0 = s.len - s.n + i0;
    } else {
      const int planes = p.B * p.Hq, runs = (p.N + p.rows_item - 1) / p.rows_item;
      if (idx >= planes * runs) return false;
      const int plane = idx % planes;
      I.row0 = I.p0 = (runs - 1 - idx / planes) * p.rows_item;
      toks = min(p.rows_item, p.N - I.p0);
      cap = TILE;
      I.b = plane / p.Hq;
      I.head0 = plane % p.Hq;
      I.kvh = I.head0 / p.g;
      I.g = 1;
      idx += gridDim.x;
    }
    I.step = cap;
    I.toks0 = min(toks, cap);
    I.toks1 = toks - I.toks0;
    I.two = I.toks1 > 0;
    I.kt = key_tiles<TILE>(I.p0, I.p0 + toks - 1, p.window, p.sinks);
    const int e0 = I.p0 + I.toks0 - 1, e1 = I.p0 + toks - 1;
    const KeyTiles k0 = key_tiles<TILE>(I.p0, e0, p.window, p.sinks);
    const KeyTiles k1 = key_tiles<TILE>(I.p0 + cap, e1, p.window, p.sinks);
    I.ns0 = k0.ns;
    I.lo0 = k0.lo;
    I.hi0 = k0.count > 0 ? e0 / TILE : -1;
    I.ns1 = k1.ns;
    I.lo1 = k1.lo;
    I.hi1 = k1.count > 0 ? e1 / TILE : -1;
    I.units = max(1, I.kt.count);
    I.off = 0;
    int take = I.units;
    if (PAGED) {
      I.off = at.off;
      take = min(left, I.units - at.off);
      left -= take;
      at.off = 0;
      if (++at.kvh == p.batch.Hkv) {
        at.kvh = 0;
        ++at.run;
        while (at.b < p.batch.seqs) {
          const Seq s = load_seq(p.batch.q_start, p.batch.kv_len, at.b, p.batch.T, p.batch.cap);
          if (at.run * p.batch.TI < s.n) break;
          at.run = 0;
          ++at.b;
        }
      }
    }
    I.cut = take < I.units;
    I.T = I.kt.count > 0 ? take : 0;
    I.seg = seg++;
    return true;
  }
};

template <int HD, bool PAGED>
__global__ void __launch_bounds__(NTHREADS, 1)
    win_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TcParams p) {
  using C = Cfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Misc& M = *reinterpret_cast<Misc*>(smem + C::OFF_MISC);
  volatile int* abort = &M.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

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
    for (int s = 0; s < 2; ++s) {
      mbar_init(&M.s_full[s], 1);
      mbar_init(&M.p_full[s], 4);
      mbar_init(&M.pv_done[s], 1);
    }
    mbar_init(&M.join_ready, 4);
    mbar_init(&M.join_done, 4);
    mbar_init(&M.drain, 1);
    M.abort = 0;
    fence_mbar_init();
  }
  if (warp == WARP_MMA) {
    tmem_alloc(&M.tmem_base, 512);
    tmem_relinquish();
  }
  if (PAGED && warp == 0) {
    const long long U = p.batch.total<TILE>();
    const long long per = share(U, (int)gridDim.x, kMinUnits);
    const long long u0 = per * blockIdx.x;
    const long long n = u0 < U ? (U - u0 < per ? U - u0 : per) : 0;
    Place at{p.batch.seqs, 0, 0, 0};
    if (n > 0) at = p.batch.locate<TILE>(u0);
    if (lane == 0) {
      M.at = at;
      M.left = (int)n;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = M.tmem_base;
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  Walk<PAGED> walk(p, M);
  Item I;
  uint32_t base = 0;  // key tiles before this item

  if (warp == WARP_TMA) {
    // ================================================================ producer
    if (lane == 0) {
      prefetch_tensormap(&tmQ);
      prefetch_tensormap(&tmK);
      prefetch_tensormap(&tmV);
    }
    uint32_t q_issued = 0, k_issued = 0, v_issued = 0;
    bool ok = true;
    while (ok && walk.next(I)) {
      if (I.T == 0) continue;
      if (q_issued > 0 && !__all_sync(0xffffffffu, mbar_wait(&M.q_empty, (q_issued - 1) & 1u, abort))) break;
      if (lane == 0) {
        const int slots = I.two ? 2 : 1;
        const uint32_t bytes = PAGED ? (uint32_t)(p.TQ * p.g * HD * 2) : (uint32_t)C::TB;
        mbar_expect_tx(&M.q_full, bytes * slots);
        for (int s = 0; s < slots; ++s)
          for (int f = 0; f < HD / 64; ++f) {
            uint8_t* dst = sQ + s * C::TB + f * C::HALF;
            if (PAGED)
              tma_load_4d(dst, &tmQ, &M.q_full, 64 * f, I.head0, I.row0 + s * p.TQ, 0);
            else
              tma_load_4d(dst, &tmQ, &M.q_full, 64 * f, I.row0 + s * TILE, p.zq & 2 ? 0 : I.head0, p.zq & 1 ? 0 : I.b);
          }
      }
      ++q_issued;
      const int pmax = I.p0 + I.toks0 + I.toks1 - 1, lo_min = I.p0 - p.window + 1;
      // One key tile: its pages, a copy per lane (a page, or its half of the columns).
      auto load = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* bar, int t, int zero, uint32_t* bad) {
        if (!PAGED) {
          if (lane == 0) {
            mbar_expect_tx(bar, C::TB);
            for (int f = 0; f < HD / 64; ++f)
              tma_load_4d(dst + f * C::HALF, map, bar, 64 * f, t * TILE, zero & 2 ? 0 : I.kvh, zero & 1 ? 0 : I.b);
          }
          return;
        }
        const int rows = min(p.page, TILE), copies = TILE / rows * (HD / 64);
        const int u = t * TILE + (lane / (HD / 64)) * rows;
        int pg = p.num_pages;  // past the end: zeros, and nothing read
        const bool seen = u <= pmax && (u + rows > lo_min || u < p.sinks);
        if (lane < copies && seen) {
          const int id = p.table[(int64_t)I.b * p.max_pages + u / p.page];
          if ((unsigned)id < (unsigned)p.num_pages) pg = id;
        }
        if (bad != nullptr) {
          const unsigned gone = __ballot_sync(0xffffffffu, lane < copies && seen && pg == p.num_pages);
          if (lane == 0) {
            uint32_t bits = 0;
            for (unsigned m = gone; m; m &= m - 1) {
              const int r = ((__ffs(m) - 1) / (HD / 64)) * rows;
              bits |= ((1u << (rows / 16)) - 1u) << (r / 16);
            }
            *bad = bits;
          }
        }
        if (lane == 0) mbar_expect_tx(bar, C::TB);
        __syncwarp();
        if (lane < copies) {
          const int f = lane % (HD / 64), r = (lane / (HD / 64)) * rows;
          tma_load_4d(dst + f * C::HALF + r * 128, map, bar, 64 * f, u % p.page, zero & 2 ? 0 : I.kvh,
                      (zero & 1) && pg < p.num_pages ? 0 : pg);
        }
        __syncwarp();
      };
      for (int j = 0; j < I.T; ++j) {
        const uint32_t n = base + j;
        const int t = I.tile(j), sk = (int)(n % C::NSK), sv = (int)(n % C::NSV);
        if (n >= C::NSK && !__all_sync(0xffffffffu, mbar_wait(&M.k_empty[sk], (n / C::NSK - 1) & 1u, abort))) {
          ok = false;
          break;
        }
        load(&tmK, sK + sk * C::TB, &M.k_full[sk], t, p.zk, &M.bad[n & 7]);
        k_issued = n + 1;
        if (n >= C::NSV && !__all_sync(0xffffffffu, mbar_wait(&M.v_empty[sv], (n / C::NSV - 1) & 1u, abort))) {
          ok = false;
          break;
        }
        load(&tmV, sV + sv * C::TB, &M.v_full[sv], t, p.zv, nullptr);
        v_issued = n + 1;
      }
      base += I.T;
    }
    // every copy must have landed before the CTA ends
    int dummy = 0;
    if (q_issued) mbar_wait(&M.q_full, (q_issued - 1) & 1u, &dummy);
    for (uint32_t n = k_issued > C::NSK ? k_issued - C::NSK : 0; n < k_issued; ++n) {
      dummy = 0;
      mbar_wait(&M.k_full[n % C::NSK], (n / C::NSK) & 1u, &dummy);
    }
    for (uint32_t n = v_issued > C::NSV ? v_issued - C::NSV : 0; n < v_issued; ++n) {
      dummy = 0;
      mbar_wait(&M.v_full[n % C::NSV], (n / C::NSV) & 1u, &dummy);
    }
  } else if (warp == WARP_MMA) {
    // ================================================================ MMA issuer (lane 0 issues)
    const uint32_t aq = smem_u32(sQ), ak = smem_u32(sK), av = smem_u32(sV);
    uint32_t items = 0, pc0 = 0, pc1 = 0;  // P tiles of each slot so far
    bool ok = true;
    while (ok && walk.next(I)) {
      if (I.T == 0) continue;
      if (!__all_sync(0xffffffffu, mbar_wait(&M.q_full, items & 1u, abort))) break;
      ++items;
      const int pmax = I.p0 + I.toks0 + I.toks1 - 1, lo_min = I.p0 - p.window + 1;
      uint32_t half_read = 0;  // key tiles (mod 32) whose first of two logit products is issued
      int nx0 = I.next(0, 0), nx1 = I.next(1, 0);
      bool started0 = false, started1 = false;
      auto issue_s = [&](int s) {
        const int j = s ? nx1 : nx0;
        const uint32_t n = base + j;
        const int sk = (int)(n % C::NSK);
        if (!__all_sync(0xffffffffu, mbar_wait(&M.k_full[sk], (n / C::NSK) & 1u, abort))) return false;
        tc_fence_after();
        const bool both = I.active(0, j) && I.active(1, j);
        const bool last = !both || ((half_read >> (j & 31)) & 1u);
        if (both) half_read ^= 1u << (j & 31);
        const int nxt = I.next(s, j + 1);
        if (s) nx1 = nxt; else nx0 = nxt;
        if (lane == 0) {
          const uint32_t q = aq + (I.two ? s * C::TB : 0);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint32_t o = (kk >> 2) * C::HALF + (kk & 3) * 32;
            mma_ss(tmem + COL_S + TILE * s, smem_desc_sw128(q + o, 16, 1024),
                   smem_desc_sw128(ak + sk * C::TB + o, 16, 1024), C::IDESC_S, kk > 0 ? 1u : 0u);
          }
          tc_commit(&M.s_full[s]);
          if (last) tc_commit(&M.k_empty[sk]);
          if (nx0 >= I.T && nx1 >= I.T) tc_commit(&M.q_empty);
        }
        __syncwarp();
        return true;
      };
      const int f = nx0 <= nx1 ? 0 : 1;
      if ((f ? nx1 : nx0) < I.T) ok = issue_s(f);
      if (ok && (f ? nx0 : nx1) < I.T) ok = issue_s(1 - f);
      for (int j = 0; ok && j < I.T; ++j) {
        const uint32_t n = base + j;
        const int sv = (int)(n % C::NSV);
        bool fixed = !PAGED;
        const bool second = I.active(1, j);
        const bool first = I.active(0, j);
        for (int s = 0; ok && s < 2; ++s) {
          if (!(s ? second : first)) continue;
          if (!__all_sync(0xffffffffu, mbar_wait(&M.v_full[sv], (n / C::NSV) & 1u, abort))) {
            ok = false;
            break;
          }
          if (!fixed) {
            // V rows that no query sees may hold anything (NaN times a zero weight is NaN): zeros instead
            const int u0 = I.tile(j) * TILE;
            if (u0 + TILE - 1 > pmax || (u0 < lo_min && u0 + TILE > p.sinks)) {
              for (int e = lane; e < TILE * (HD / 64) * 8; e += 32) {
                const int r = (e >> 3) % TILE, u = u0 + r;
                if (u > pmax || (u < lo_min && u >= p.sinks))
                  *reinterpret_cast<uint4*>(sV + sv * C::TB + (e >> 3) / TILE * C::HALF + r * 128 + (e & 7) * 16) =
                      make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
            fixed = true;
          }
          if (!__all_sync(0xffffffffu, mbar_wait(&M.p_full[s], (s ? pc1 : pc0) & 1u, abort))) {
            ok = false;
            break;
          }
          if (s) ++pc1; else ++pc0;
          tc_fence_after();
          if (lane == 0) {
#pragma unroll
            for (int kk = 0; kk < TILE / 16; ++kk)
              mma_ts(tmem + HD * s, tmem + COL_S + TILE * s + 64 + 8 * kk,
                     smem_desc_sw128(av + sv * C::TB + kk * 2048, C::HALF, 1024), C::IDESC_PV,
                     ((s ? started1 : started0) || kk > 0) ? 1u : 0u);
            tc_commit(&M.pv_done[s]);
            if (s == 1 || !second) tc_commit(&M.v_empty[sv]);
          }
          __syncwarp();
          if (s) started1 = true; else started0 = true;
          if ((s ? nx1 : nx0) < I.T) ok = issue_s(s);
        }
      }
      base += I.T;
    }
    if (lane == 0) {
      tc_commit(&M.drain);
      int dummy = 0;
      mbar_wait(&M.drain, 0, &dummy);
    }
    __syncwarp();
  } else {
    // ================================================================ softmax
    const int s = warp >> 2;
    const int row = (warp & 3) * 32 + lane;  // row of the slot == TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_base + COL_S + TILE * s, o_addr = lane_base + HD * s;
    uint32_t sc = 0, joins = 0;  // logit tiles and joined items so far
    bool ok = true;
    while (ok && walk.next(I)) {
      const int g = I.g;
      const int nrows = (s && I.two ? I.toks1 : I.toks0) * g;
      const int pbase = I.p0 + (s && I.two ? I.step : 0);
      const int pos = pbase + row / g;
      const int r0 = (warp & 3) * 32, rlast = min(r0 + 31, nrows - 1);
      const bool live = r0 < nrows;  // the warp holds rows
      const int wmin = pbase + r0 / g, wmax = pbase + rlast / g;
      float m = kNegInf, l = 0.f;
      int steps = 0;
      for (int j = 0; j < I.T; ++j) {
        if (!I.active(s, j)) continue;
        if (!__all_sync(0xffffffffu, mbar_wait(&M.s_full[s], sc & 1u, abort))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (live) {
          const int u0 = I.tile(j) * TILE;
          const uint32_t bad = PAGED ? M.bad[(base + j) & 7] : 0u;
          const bool none = u0 > wmax || (u0 + TILE - 1 <= wmin - p.window && u0 >= p.sinks);
          const bool all = u0 + TILE - 1 <= wmin && (u0 > wmax - p.window || u0 + TILE <= p.sinks) && bad == 0;
          // 64 logits at a time stay in registers: the first half is read for its maximum and once
          // more for its weights, the second half once.
          float x[64];
          auto load_half = [&](int q) {
            tmem_ld32(s_addr + 64 * q, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
            tmem_ld32(s_addr + 64 * q + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
            tmem_wait_ld();
            if (!all) {
              const int v0 = u0 + 64 * q;
              const int hi = pos - v0, lo = pos - p.window - v0, sk = p.sinks - v0;  // sees lo < c <= hi, or c < sk
              const uint32_t gone = bad >> (4 * q);
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (c > hi || (c <= lo && c >= sk) || ((gone >> (c >> 4)) & 1u)) x[c] = kNegInf;
            }
          };
          float a0 = kNegInf, a1 = kNegInf, a2 = kNegInf, a3 = kNegInf;
          if (!none) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              load_half(q);
#pragma unroll
              for (int c = 0; c < 64; c += 4) {
                a0 = fmaxf(a0, x[c]);
                a1 = fmaxf(a1, x[c + 1]);
                a2 = fmaxf(a2, x[c + 2]);
                a3 = fmaxf(a3, x[c + 3]);
              }
            }
          }
          const float mx = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)) * p.c;  // scale > 0
          // Raise the running maximum when the tile exceeds it by more than the threshold; O (after the
          // previous P V) and the sum are then rescaled.
          const bool need = m != kNegInf && mx > m + kRescaleThreshold;
          if (__any_sync(0xffffffffu, need)) {
            if (!__all_sync(0xffffffffu, mbar_wait(&M.pv_done[s], (sc - 1) & 1u, abort))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const float f = need ? ex2(m - mx) : 1.0f;
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 16) {
              uint32_t r[16];
              tmem_ld16(o_addr + c0, r);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * f);
              tmem_st16(o_addr + c0, r);
            }
            if (need) {
              l *= f;
              m = mx;
            }
          }
          if (m == kNegInf) m = mx;
          const float nm = m == kNegInf ? 0.f : -m;
          uint32_t pk[32];
          if (none) {
#pragma unroll
            for (int c = 0; c < 32; ++c) pk[c] = 0u;
            tmem_st32(s_addr + 64, pk);
            tmem_st32(s_addr + 96, pk);
          } else {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int q = 1; q >= 0; --q) {
              if (q == 0) load_half(0);
#pragma unroll
              for (int c = 0; c < 64; c += 2) {
                const float e0 = ex2(fmaf(x[c], p.c, nm));
                const float e1 = ex2(fmaf(x[c + 1], p.c, nm));
                s0 += e0;
                s1 += e1;
                pk[c / 2] = pack_bf16(e0, e1);
              }
              tmem_st32(s_addr + 64 + 32 * q, pk);
            }
            l += s0 + s1;
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M.p_full[s]);
        ++sc;
        ++steps;
      }
      if (!ok) break;
      base += I.T;

      // ---- epilogue of the item
      if (steps > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(&M.pv_done[s], (sc - 1) & 1u, abort))) break;
        tc_fence_after();
      }
      const bool join = !I.two && I.T > 1;
      if (join && s == 1) {
        M.jm[row] = m;
        M.jl[row] = l;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M.join_ready);
        if (!__all_sync(0xffffffffu, mbar_wait(&M.join_done, joins & 1u, abort))) break;
        ++joins;
        tc_fence_after();
        continue;
      }
      if (!I.two && s == 1) continue;
      float f0 = 1.f, f1 = 0.f;
      if (join) {
        if (!__all_sync(0xffffffffu, mbar_wait(&M.join_ready, joins & 1u, abort))) break;
        tc_fence_after();
        const float m1 = M.jm[row], l1 = M.jl[row], mm = fmaxf(m, m1);
        f0 = m == kNegInf ? 0.f : ex2(m - mm);
        f1 = m1 == kNegInf ? 0.f : ex2(m1 - mm);
        l = l * f0 + l1 * f1;
        m = mm;
      }
      if (live) {
        const bool mine = row < nrows;
        const bool cut = PAGED && I.cut;
        const float inv = cut ? 1.f : (l == 0.f ? 0.f : 1.0f / l);
        f0 *= inv;
        f1 *= inv;
        const int tok = I.row0 + (s && I.two ? I.step : 0) + row / g, head = I.head0 + row % g;
        float* po = nullptr;
        bf16* ho = nullptr;
        if (mine) {
          if (cut) {
            float* pb = p.part + (size_t)(2 * blockIdx.x + (I.seg ? 1 : 0)) * partial_floats(2 * TILE, HD);
            const int pr = (s && I.two ? I.step * g : 0) + row;
            po = pb + (size_t)pr * HD;
            pb[2 * TILE * HD + pr] = m;
            pb[2 * TILE * HD + 2 * TILE + pr] = l;
          } else {
            ho = row_ptr_w<bf16>(p.h, PAGED ? 0 : I.b, head, tok);
            const int64_t o = PAGED ? (int64_t)head * p.batch.T + tok : ((int64_t)I.b * p.Hq + head) * p.N + tok;
            p.lse[o] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
          }
        }
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 32) {
          float o[32];
          uint32_t r[32];
          if (steps > 0) {
            tmem_ld32(o_addr + c0, r);
            tmem_wait_ld();
          }
          // a row without weight stays zero whatever the accumulator holds
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = steps > 0 && f0 != 0.f ? __uint_as_float(r[c]) * f0 : 0.f;
          if (join) {
            tmem_ld32(o_addr + HD + c0, r);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] += f1 != 0.f ? __uint_as_float(r[c]) * f1 : 0.f;
          }
          if (po != nullptr) {
#pragma unroll
            for (int c = 0; c < 32; c += 4)
              *reinterpret_cast<float4*>(po + c0 + c) = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
          } else if (ho != nullptr) {
            uint4* dst = reinterpret_cast<uint4*>(ho + c0);
#pragma unroll
            for (int v = 0; v < 4; ++v)
              dst[v] = make_uint4(pack_bf16(o[8 * v], o[8 * v + 1]), pack_bf16(o[8 * v + 2], o[8 * v + 3]),
                                  pack_bf16(o[8 * v + 4], o[8 * v + 5]), pack_bf16(o[8 * v + 6], o[8 * v + 7]));
          }
        }
      }
      if (join) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M.join_done);
        ++joins;
      }
    }
  }

  // ---- tear-down
  tc_fence_before();
  __syncthreads();
  if (M.abort && threadIdx.x == 0) atomicCAS(p.status, 0, (int)SSA_ERR_TIMEOUT);
  if (warp == WARP_MMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD>
constexpr int smem_bytes() {
  return Cfg<HD>::OFF_MISC + (int)sizeof(Misc) + 1024;
}
static_assert(smem_bytes<128>() <= 232448, "shared memory of a CTA");

template <int HD, bool PAGED>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const TcParams& p, int ctas,
                   cudaStream_t st) {
  auto kern = win_fwd_tc_kernel<HD, PAGED>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<HD>());
  if (e != cudaSuccess) return e;
  kern<<<ctas, NTHREADS, smem_bytes<HD>(), st>>>(q, k, v, p);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_win_fwd_tc(const WinDims& D, const WinFwdArgs& a, int32_t* status, cudaStream_t st) {
  CUtensorMap q, k, v;
  TcParams p{};
  if (!win_tma_map(&q, a.q, D.B, D.Hq, D.N, TILE, D.d, &p.zq) || !win_tma_map(&k, a.k, D.B, D.Hkv, D.N, TILE, D.d, &p.zk) ||
      !win_tma_map(&v, a.v, D.B, D.Hkv, D.N, TILE, D.d, &p.zv))
    return cudaErrorInvalidValue;
  p.h = a.h;
  p.lse = a.lse;
  p.status = status;
  p.B = D.B;
  p.Hq = D.Hq;
  p.g = D.g;
  p.N = D.N;
  p.window = D.window;
  p.sinks = D.sinks;
  p.c = D.scale * kLog2e;
  const int64_t planes = (int64_t)D.B * D.Hq;
  p.rows_item = planes * ((D.N + 255) / 256) >= kCtas ? 256 : 128;
  const int64_t items = planes * ((D.N + p.rows_item - 1) / p.rows_item);
  const int ctas = (int)(items < kCtas ? items : kCtas);
  return D.d == 64 ? launch<64, false>(q, k, v, p, ctas, st) : launch<128, false>(q, k, v, p, ctas, st);
}

size_t paged_tc_ws_bytes(const PagedDims& D) {
  return ((size_t)2 * kCtas * partial_floats(2 * TILE, D.d) * 4 + 255) / 256 * 256;
}

cudaError_t launch_paged_tc(const PagedDims& D, const PagedArgs& a, int32_t* status, cudaStream_t st) {
  CUtensorMap q, k, v;
  TcParams p{};
  p.TQ = TILE / D.g;
  const int rows = D.page < TILE ? D.page : TILE;
  // Packed queries: (column, head, token); a box holds the group's heads of TQ tokens, token-major.
  if (!tma_map_4d(&q, a.q.p, D.d, D.Hq, D.T, 1, D.Hq > 1 ? a.q.sh : 8, D.T > 1 ? a.q.sn : 8, 8, D.g, p.TQ) ||
      !win_tma_map(&k, a.k, D.num_pages, D.Hkv, D.page, rows, D.d, &p.zk) ||
      !win_tma_map(&v, a.v, D.num_pages, D.Hkv, D.page, rows, D.d, &p.zv))
    return cudaErrorInvalidValue;
  p.h = a.h;
  p.lse = a.lse;
  p.status = status;
  p.Hq = D.Hq;
  p.g = D.g;
  p.window = D.window;
  p.sinks = D.sinks;
  p.c = D.scale * kLog2e;
  p.table = a.table;
  p.page = D.page;
  p.num_pages = D.num_pages;
  p.max_pages = D.max_pages;
  p.batch = Batch{a.q_start, a.kv_len, D.seqs, D.T, D.max_pages * D.page, 2 * p.TQ, D.window, D.sinks, D.Hkv};
  p.part = static_cast<float*>(a.ws);
  cudaError_t e = D.d == 64 ? launch<64, true>(q, k, v, p, kCtas, st) : launch<128, true>(q, k, v, p, kCtas, st);
  if (e != cudaSuccess) return e;
  return launch_paged_join<TILE, 2 * TILE>(D, a, kCtas, 2 * p.TQ, kMinUnits, st);
}

}  // namespace ssa
