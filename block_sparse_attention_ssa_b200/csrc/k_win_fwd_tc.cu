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
// (TMEM lanes).  Key tiles of 128 keys are shared by both slots; a step is half a tile, 64
// keys.  Warps 4 (2 s + h) .. + 3 hold the softmax of half h of slot s's tiles, warps 16 and 19
// load Q with K and V by TMA (a tile of 16-token pages is 32 copies, more than one warp issues
// in a tile's time at full memory rate), one thread of warps 17 and 18 issues the products of slot 0 and slot 1 (one issuer
// for both spent more cycles on its control flow than the products take).  TMEM: O of slot s
// at HD s, its two S buffers of 64 columns at 256 + 128 s; P (bf16 pairs) overwrites the second
// half of its S buffer and feeds P V from TMEM.  The next tile's logits are issued behind P V
// of the same half, so they are ready when the softmax warps come to them.
// A row's two softmax threads share one running maximum: a step's thread takes the one that
// the step before published, publishes its own before it forms any exponential, and keeps its
// own sum, so that only the maxima form a chain and four warps per scheduler hide the latency
// of the exponentials (with one thread per row and two warps the schedulers issued in 35 % of
// the cycles and a tile of both slots took 4200 of them).
// An item whose rows fit one slot gives the odd key tiles to slot 1 with the same queries,
// and slot 0's warps join the two softmaxes at the end, so that a decoding step has four
// chains in flight too.
//
// Rows.  Window form: a row is a token of one query head.  Paged form: a row is a
// (new token, head of the group) pair, so the g heads of a kv head share each K/V load
// and a single token fills g rows; 128 / g tokens to a slot.  Paged items are cut into
// equal shares of key tiles (win_common.cuh); cut items leave fp32 partials.
//
// Measured (bf16, 32 heads over 8, d = 128).  32768 tokens, window 1024, 64 sinks: 635 us, 905 TFLOP/s of visible pairs
// (20 passes from idle; 736 in long runs).  Chunks of 896 to 2048 tokens (5888 in all) over 6125 to 14000 more, 4 sequences:
// 1075 us, 1051 TFLOP/s (1233 in long runs).
// Bound by the chain of a step, 3500 cycles for a tile of both slots: logits waited for 1100, loaded for their maximum 350,
// maximum passed on 570, exponentials 1200 (2048 of their pipe's cycles for both slots), P stored 330.  Over the kernel the
// tensor pipe is active 45 % of the time, the exponentials' pipe 46 % (16384 tokens, window 1024).  Between items
// 5500 cycles (sums, last product, output), which bounds short windows: 8192 tokens, 32 heads over 2, d = 64, window 256:
// 77 us, 233 TFLOP/s.  One token of 64 sequences over 2094 to 8001 (323040 in all, 1.32 GB): 239 us, 5.5 TB/s, bound by
// memory.  The runs of a sequence are counted one by one (win_common.cuh): 32768 new tokens, 32 heads over 2, d = 64,
// window 256, take 1203 us, as many tokens of the window form 279.
#include "win_rows.cuh"

#include "sm100_ptx.cuh"

namespace ssa {
namespace {

using namespace sm100;
using bf16 = __nv_bfloat16;

constexpr int TILE = 128;
constexpr int UNIT = 64;  // keys of a step
constexpr int NTHREADS = 640;
constexpr int WARP_TMA = 16, WARP_MMA = 17, WARP_TMA_V = 19;  // and WARP_MMA + 1 for slot 1

constexpr int kCtas = 148;     // one per SM
constexpr float kRescaleThreshold = 8.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t COL_S = 256;

template <int HD, bool PAGED>
struct Cfg {
  // K, V tiles in flight.  At d = 128 the paged form fills shared memory: one token of 64 sequences takes 236 us with three
  // K tiles, 244 to 254 with two; the window form does better with two (32768 tokens, window 1024: 647 us against 660).
  static constexpr int NSK = HD == 128 ? (PAGED ? 3 : 2) : 4, NSV = HD == 128 ? 2 : 4;
  static constexpr int TB = TILE * HD * 2;
  static constexpr int HALF = TILE * 128;  // 64 columns of a tile: 128 rows of 128 bytes
  static constexpr int OFF_K = 2 * TB, OFF_V = OFF_K + NSK * TB, OFF_MISC = OFF_V + NSV * TB;
  static constexpr uint32_t IDESC_S = idesc_bf16_f32(TILE, UNIT, false, false);
  static constexpr uint32_t IDESC_PV = idesc_bf16_f32(TILE, HD, false, true);
};

struct Misc {
  uint64_t q_full, q_empty, k_full[4], k_empty[4], v_full[4], v_empty[4];
  // by half: who waits for a step knows the same half's step before done, and a barrier tells only
  // neighbouring phases apart
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];
  uint64_t m_ready[2][2][4];        // a warp's running maxima are published
  uint64_t sum_ready[2][4], total_ready[2][4];
  uint64_t o_free[2];               // O of the slot has been read
  uint64_t join_ready, join_done, drain[2];
  uint32_t tmem_base;
  int abort;
  int turn;  // 1 while an issuer feeds the tensor core
  int left;
  int again;  // rows that are not finite were stored
  Place at;
  uint32_t bad[8];  // pages missing from a key tile, a bit per 16 keys (ring of 2 NSK tiles)
  float mref[2][TILE];  // running maximum of each row
  float sum[2][TILE];   // at an item's end: the first half's sum, then the whole one
};

struct TcParams {
  TensorRef q, k, v, h;
  float* lse;
  int32_t* status;
  int B, Hq, g, N, window, sinks;
  int zk, zv, zq;    // broadcast dimensions of K, V, Q: bit 0 batch, bit 1 head
  int rows_item;     // window form: tokens of an item (256, or 128 when those would be fewer than the SMs)
  float c;           // scale * log2(e)
  bool wide;         // h in 32-byte pieces
  // paged form
  const int32_t* table;
  Batch batch;
  int page, num_pages, max_pages, TQ;
  float* part;
};

// One work item as a role of slot s sees it.
struct Item {
  int b, kvh, head0, row0, p0, g;  // row0: first token (window) or packed row (paged); p0: its position
  int toks, toks0;                 // tokens of the item and of slot 0
  int T, off, seg, units;          // key tiles of this CTA's share, the first one's index
  bool two, cut;                   // both slots hold rows; share of an item only
  KeyTiles kt;
  // Two slots of rows: the slot uses the share's tiles j < A and B <= j < E (its sinks, its window),
  // the other one j < oA and oB <= j < oE; every tile is used by one of them.  Alone, the slots take
  // the tiles in turn.
  int s, A, B, E, oA, oB, oE;
  __device__ __forceinline__ int tile(int j) const { return kt.tile(off + j); }
  __device__ __forceinline__ bool shared(int j) const { return two && (j < oA || (j >= oB && j < oE)); }
  __device__ __forceinline__ int next(int j) const {  // the slot's first tile at or after j (T: none)
    if (!two) return min(j + ((j ^ s) & 1), T);
    if (j >= A) {
      j = max(j, B);
      if (j >= E) j = T;
    }
    return min(j, T);
  }
};

// Waits (bounded) until the other issuer has left the tensor core's queue.
__device__ __forceinline__ bool take_turn(Misc& M, volatile int* abort) {
  if (atomicCAS(&M.turn, 0, 1) == 0) return true;
  const long long t0 = clock64();
  while (atomicCAS(&M.turn, 0, 1) != 0) {
    if (*abort) return false;
    if (clock64() - t0 > kWaitCycles) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void pass_turn(Misc& M) { atomicExch(&M.turn, 0); }

// The CTA's items in order.
template <bool PAGED>
struct Walk {
  const TcParams& p;
  Place at;
  int left, idx, seg, s;
  __device__ Walk(const TcParams& p_, const Misc& M, int s_) : p(p_), at(M.at), left(M.left), idx(blockIdx.x), seg(0), s(s_) {}

  __device__ bool next(Item& I) {
    int toks, cap, seq_n = 0;
    if (PAGED) {
      if (left <= 0 || at.b >= p.batch.seqs) return false;
      const Seq q = load_seq(p.batch.q_start, p.batch.kv_len, at.b, at.q0, p.batch.T, p.batch.cap);
      const int i0 = at.run * p.batch.TI;
      toks = min(p.batch.TI, q.n - i0);
      seq_n = q.n;
      cap = p.TQ;
      I.b = at.b;
      I.kvh = at.kvh;
      I.head0 = at.kvh * p.g;
      I.g = p.g;
      I.row0 = q.q0 + i0;
      I.p0 = q.len - q.n + i0;
    } else {
      const int planes = p.B * p.Hq, runs = (p.N + p.rows_item - 1) / p.rows_item;
      if (idx >= planes * runs) return false;
      const int run = idx / planes, plane = idx - run * planes;
      I.row0 = I.p0 = (runs - 1 - run) * p.rows_item;
      toks = min(p.rows_item, p.N - I.p0);
      cap = TILE;
      I.b = plane / p.Hq;
      I.head0 = plane - I.b * p.Hq;
      I.kvh = I.head0 / p.g;
      I.g = 1;
      idx += gridDim.x;
    }
    I.s = s;
    I.toks = toks;
    I.toks0 = min(toks, cap);
    I.two = toks > cap;
    I.kt = key_tiles<TILE>(I.p0, I.p0 + toks - 1, p.window, p.sinks);
    I.units = max(1, I.kt.count);
    I.off = 0;
    int take = I.units;
    if (PAGED) {
      I.off = at.off;
      take = min(left, I.units - at.off);
      left -= take;
      at.off = 0;
      if (left > 0 && ++at.kvh == p.batch.Hkv) {
        at.kvh = 0;
        if (++at.run * p.batch.TI >= seq_n) {
          at.run = 0;
          at.q0 += seq_n;
          at.b = p.batch.next_seq<1>(at.b + 1, at.q0);
        }
      }
    }
    auto own = [&](int first, int last, int& A, int& B, int& E) {
      const KeyTiles k = key_tiles<TILE>(first, last, p.window, p.sinks);
      A = (k.ns > I.kt.lo ? I.kt.ns + k.ns - I.kt.lo : k.ns) - I.off;
      B = I.kt.ns + k.lo - I.kt.lo - I.off;
      E = k.count > 0 ? I.kt.ns + last / TILE - I.kt.lo + 1 - I.off : 0;
    };
    const int f = s ? cap : 0, e = s ? toks : I.toks0;  // tokens of the slot and of the other one
    own(I.p0 + f, I.p0 + e - 1, I.A, I.B, I.E);
    own(I.p0 + cap - f, I.p0 + toks + I.toks0 - e - 1, I.oA, I.oB, I.oE);
    I.cut = take < I.units;
    I.T = I.kt.count > 0 ? take : 0;
    I.seg = seg++;
    return true;
  }
};

// The CTA's rows that are not finite once more (win_rows.cuh), a warp a row.  Behind the loop over the items, so that nothing
// of it is held in registers there (within it, 270 to 530 bytes were spilled), and inline: a function called there
// took 2 us of every launch (8192 tokens, window 256: 79.6 us, inline 77.5, without any of it 77.8).
template <int HD, bool PAGED>
__device__ __forceinline__ void form_again(const TcParams& p, const Misc& M) {
  Walk<PAGED> walk(p, M, 0);
  Item I;
  while (walk.next(I)) {
    if (I.T == 0) continue;
    const KeyRows<bf16> keys{p.k, p.v, I.b, I.kvh, PAGED ? p.table : nullptr, p.page, p.num_pages, p.max_pages};
    for (int r = threadIdx.x >> 5; r < I.toks * I.g; r += NTHREADS / 32) {
      const int i = PAGED ? r / I.g : r, tok = I.row0 + i, head = I.head0 + (PAGED ? r % I.g : 0);
      const RowView view{I.kt, I.p0 + i, I.off, I.off + I.T, p.window, p.sinks, p.N};
      RowOut<bf16> o{};
      if (PAGED && I.cut) {
        float* pb = p.part + (size_t)(2 * blockIdx.x + (I.seg ? 1 : 0)) * partial_floats(2 * TILE, HD);
        o.part = pb + (size_t)r * HD;
        o.m = pb + 2 * TILE * HD + r;
        o.l = o.m + 2 * TILE;
      } else {
        o.out = row_ptr_w<bf16>(p.h, PAGED ? 0 : I.b, head, tok);
        o.lse = p.lse + (PAGED ? (int64_t)head * p.batch.T + tok : ((int64_t)I.b * p.Hq + head) * p.N + tok);
      }
      mend_row<bf16, HD, TILE>(keys, view, row_ptr<bf16>(p.q, PAGED ? 0 : I.b, head, tok), o, p.c);
    }
  }
}

template <int HD, bool PAGED>
__global__ void __launch_bounds__(NTHREADS, 1)
    win_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmVs,
                      const __grid_constant__ TcParams p) {
  using C = Cfg<HD, PAGED>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;  // tiles need 1024-byte alignment: checked below
  Misc& M = *reinterpret_cast<Misc*>(smem + C::OFF_MISC);
  volatile int* abort = &M.abort;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform

  if (smem_u32(smem_raw) & 1023u) {  // no room for slack: shared memory starts on a 1024-byte boundary
    if (threadIdx.x == 0) atomicCAS(p.status, 0, (int)SSA_ERR_CUDA);
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(&M.q_full, 1);
    mbar_init(&M.q_empty, 2);
    for (int i = 0; i < C::NSK; ++i) {
      mbar_init(&M.k_full[i], 1);
      mbar_init(&M.k_empty[i], 2);  // each slot's issuer, or the only user of the tile twice
    }
    for (int i = 0; i < C::NSV; ++i) {
      mbar_init(&M.v_full[i], 1);
      mbar_init(&M.v_empty[i], 2);
    }
    for (int s = 0; s < 2; ++s) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&M.s_full[s][i], 1);
        mbar_init(&M.p_full[s][i], 4);
        mbar_init(&M.pv_done[s][i], 1);
        for (int w = 0; w < 4; ++w) mbar_init(&M.m_ready[s][i][w], 1);
      }
      for (int w = 0; w < 4; ++w) {
        mbar_init(&M.sum_ready[s][w], 1);
        mbar_init(&M.total_ready[s][w], 1);
      }
      mbar_init(&M.o_free[s], 8);
      mbar_init(&M.drain[s], 1);
    }
    mbar_init(&M.join_ready, 8);
    mbar_init(&M.join_done, 8);
    M.abort = 0;
    M.turn = 0;
    M.again = 0;
    fence_mbar_init();
  }
  if (warp == WARP_MMA) {
    tmem_alloc(&M.tmem_base, 512);
    tmem_relinquish();
  }
  if (PAGED && warp == 0) {
    bool falls;
    const long long U = p.batch.total<TILE>(falls);
    const long long per = share(U, (int)gridDim.x);
    const long long u0 = per * blockIdx.x;
    const long long n = u0 < U ? (U - u0 < per ? U - u0 : per) : 0;
    Place at{p.batch.seqs, 0, 0, 0, 0};
    if (n > 0) at = p.batch.locate<TILE>(u0, falls);
    if (lane == 0) {
      M.at = at;
      M.left = (int)n;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (PAGED) allow_ahead();  // the join
  const uint32_t tmem = M.tmem_base;
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  Walk<PAGED> walk(p, M, warp < WARP_TMA ? warp >> 3 : (warp == WARP_MMA + 1 ? 1 : 0));
  Item I;
  uint32_t base = 0;  // key tiles before this item

  if (warp == WARP_TMA || warp == WARP_TMA_V) {
    // ================================================================ producers: Q and K, and V
    const bool is_k = warp == WARP_TMA;
    const CUtensorMap* map = is_k ? &tmK : &tmV;
    const int zero = is_k ? p.zk : p.zv, stages = is_k ? C::NSK : C::NSV;
    uint64_t* full = is_k ? M.k_full : M.v_full;
    uint64_t* empty = is_k ? M.k_empty : M.v_empty;
    uint8_t* ring = is_k ? sK : sV;
    if (lane == 0) {
      prefetch_tensormap(map);
      if (is_k) prefetch_tensormap(&tmQ);
    }
    uint32_t q_issued = 0, issued = 0;
    bool ok = true;
    while (ok && walk.next(I)) {
      if (I.T == 0) continue;
      if (is_k) {
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
      }
      const int pmax = I.p0 + I.toks - 1, lo_min = I.p0 - p.window + 1;
      for (int j = 0; j < I.T; ++j) {
        const uint32_t n = base + j;
        const int t = I.tile(j), st = (int)(n % stages);
        const uint32_t use = n / stages;
        // Pages of the tile: a copy a lane (a page, or its half of the columns).  Ids are read before the wait.
        const int rows = PAGED ? min(p.page, TILE) : TILE, copies = TILE / rows * (HD / 64);
        const int u = t * TILE + (lane / (HD / 64)) * rows;
        int pg = p.num_pages;  // past the end: zeros, and nothing read
        bool seen = false;
        if (PAGED && lane < copies) {
          seen = u <= pmax && (u + rows > lo_min || u < p.sinks);
          if (seen) {
            const int id = p.table[(int64_t)I.b * p.max_pages + u / p.page];
            if ((unsigned)id < (unsigned)p.num_pages) pg = id;
          }
        }
        if (use > 0 && !__all_sync(0xffffffffu, mbar_wait(&empty[st], (use - 1) & 1u, abort))) {
          ok = false;
          break;
        }
        uint8_t* dst = ring + st * C::TB;
        if (PAGED) {
          if (is_k) {
            const unsigned gone = __ballot_sync(0xffffffffu, seen && pg == p.num_pages);
            if (lane == 0) {
              uint32_t bits = 0;
              for (unsigned m = gone; m; m &= m - 1) {
                const int r = ((__ffs(m) - 1) / (HD / 64)) * rows;
                bits |= ((1u << (rows / 16)) - 1u) << (r / 16);
              }
              M.bad[n & 7] = bits;
            }
          }
          if (lane == 0) mbar_expect_tx(&full[st], C::TB);
          __syncwarp();
          if (lane < copies) {
            const int f = lane % (HD / 64), r = (lane / (HD / 64)) * rows;
            tma_load_4d(dst + f * C::HALF + r * 128, map, &full[st], 64 * f, u % p.page, zero & 2 ? 0 : I.kvh,
                        (zero & 1) && pg < p.num_pages ? 0 : pg);
          }
          __syncwarp();
        } else if (lane == 0) {
          // No query of the item sees more of a sink tile's keys than the sinks: V through a map that ends there, zeros
          // behind it, so that what those rows hold does not reach every later token.
          const CUtensorMap* mp = !is_k && j < I.kt.ns ? &tmVs : map;
          mbar_expect_tx(&full[st], C::TB);
          for (int f = 0; f < HD / 64; ++f)
            tma_load_4d(dst + f * C::HALF, mp, &full[st], 64 * f, t * TILE, zero & 2 ? 0 : I.kvh, zero & 1 ? 0 : I.b);
        }
        issued = n + 1;
      }
      base += I.T;
    }
    // every copy must have landed before the CTA ends
    int dummy = 0;
    if (q_issued) mbar_wait(&M.q_full, (q_issued - 1) & 1u, &dummy);
    for (uint32_t n = issued > (uint32_t)stages ? issued - stages : 0; n < issued; ++n) {
      dummy = 0;
      mbar_wait(&full[n % stages], (n / stages) & 1u, &dummy);
    }
  } else if (warp == WARP_MMA || warp == WARP_MMA + 1) {
    // ================================================================ MMA issuer of slot s
    if (elect_one()) {
      const int s = warp - WARP_MMA;
      const uint32_t aq = desc_lo(smem_u32(sQ), 16), ak = desc_lo(smem_u32(sK), 16), av = desc_lo(smem_u32(sV), C::HALF);
      const uint32_t cS = tmem + COL_S + TILE * s, cO = tmem + HD * s;
      uint32_t items = 0, np = 0, outs = 0;  // items, tiles and items with tiles of the slot so far
      bool ok = true;
      // Logits of a tile's half, and P V of it.
      auto logits = [&](uint32_t q, uint32_t k, int half) {
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint32_t o = ((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4;
          mma_ss_lo(cS + UNIT * half, q + o, k + half * (UNIT * 128 >> 4) + o, C::IDESC_S, kk > 0 ? 1u : 0u);
        }
        tc_commit(&M.s_full[s][half]);
      };
      auto weighted = [&](uint32_t v, int half, uint32_t acc) {
#pragma unroll
        for (int kk = 0; kk < UNIT / 16; ++kk)
          mma_ts_lo(cO, cS + UNIT * half + 32 + 8 * kk, v + (4 * half + kk) * 128, C::IDESC_PV, kk > 0 ? 1u : acc);
        tc_commit(&M.pv_done[s][half]);
      };
      auto release = [&](uint64_t* bar, int j) {
        tc_commit(bar);
        if (!I.shared(j)) tc_commit(bar);
      };
      while (ok && walk.next(I)) {
        if (I.T == 0) continue;
        if (!mbar_wait(&M.q_full, items & 1u, abort)) break;
        ++items;
        const uint32_t q = aq + (I.two ? s * (C::TB >> 4) : 0);
        int j = I.next(0);
        if (j < I.T) {
          const uint32_t n = base + j, sk = n % C::NSK;
          if (!(ok = mbar_wait(&M.k_full[sk], (n / C::NSK) & 1u, abort))) break;
          tc_fence_after();
          logits(q, ak + sk * (C::TB >> 4), 0);
          logits(q, ak + sk * (C::TB >> 4), 1);
          release(&M.k_empty[sk], j);
        } else {
          mbar_arrive(&M.q_empty);  // no tile of this share is the slot's
        }
        if (j < I.T) {  // the item before has read O by the time this one's first P V is due
          if (outs > 0 && !(ok = mbar_wait(&M.o_free[s], (outs - 1) & 1u, abort))) break;
          ++outs;
        }
        for (uint32_t acc = 0; j < I.T; acc = 1) {
          const int nj = I.next(j + 1);
          const uint32_t n = base + j, sv = n % C::NSV, nn = base + nj, sk = nn % C::NSK;
          const uint32_t v = av + sv * (C::TB >> 4), k = ak + sk * (C::TB >> 4);
          if (nj >= I.T) tc_commit(&M.q_empty);  // the last logits are issued
          if (!(ok = mbar_wait(&M.v_full[sv], (n / C::NSV) & 1u, abort) && mbar_wait(&M.p_full[s][0], np & 1u, abort))) break;
          const bool more = nj < I.T;
          auto k_there = [&] { return !more || mbar_wait(&M.k_full[sk], (nn / C::NSK) & 1u, abort); };
          if (I.two) {
            // P V of a half and the next logits of that half go in one piece: interleaved with the other slot's,
            // all four softmax groups would wait for one another's products and then work side by side while
            // the tensor core idles.  Everything awaited is there before the turn is taken.
            if (!(ok = k_there() && take_turn(M, abort))) break;
            tc_fence_after();
            weighted(v, 0, acc);
            if (more) logits(q, k, 0);
            pass_turn(M);
            if (!(ok = mbar_wait(&M.p_full[s][1], np & 1u, abort) && take_turn(M, abort))) break;
            tc_fence_after();
            weighted(v, 1, 1u);
            if (more) logits(q, k, 1);
            pass_turn(M);
          } else {
            // Few rows: bound by the loads, so V is released as early as its P allows, whether or not the
            // next K has arrived.
            tc_fence_after();
            weighted(v, 0, acc);
            if (!(ok = mbar_wait(&M.p_full[s][1], np & 1u, abort))) break;
            tc_fence_after();
            weighted(v, 1, 1u);
          }
          release(&M.v_empty[sv], j);
          if (more && !I.two) {
            if (!(ok = k_there())) break;
            tc_fence_after();
            logits(q, k, 0);
            logits(q, k, 1);
          }
          if (more) release(&M.k_empty[sk], nj);
          ++np;
          j = nj;
        }
        base += I.T;
      }
      tc_commit(&M.drain[s]);
      int dummy = 0;
      mbar_wait(&M.drain[s], 0, &dummy);
    }
    __syncwarp();
  } else if (warp < WARP_TMA) {
    // ================================================================ softmax
    const int s = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
    const int row = quarter * 32 + lane;  // row of the slot == TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_addr = lane_base + COL_S + TILE * s + UNIT * half;
    float* mref = &M.mref[s][row];
    // V rows that no query of the item sees may hold anything (NaN times a zero weight is NaN): zeros in
    // shared memory instead, before this slot's weights go to the product.  Both slots may write them.
    auto clear_v = [&](const Item& I, uint32_t n, int u0) {
      const int pmax = I.p0 + I.toks - 1, lo_min = I.p0 - p.window + 1;
      if (!mbar_wait(&M.v_full[n % C::NSV], (n / C::NSV) & 1u, abort)) return;  // noticed at the next wait
      uint8_t* sv = sV + (n % C::NSV) * C::TB;
      for (int e = threadIdx.x & 127; e < TILE * (HD / 64) * 8; e += 128) {
        const int r = (e >> 3) % TILE, u = u0 + r;
        if (u > pmax || (u < lo_min && u >= p.sinks))
          *reinterpret_cast<uint4*>(sv + (e >> 3) / TILE * C::HALF + r * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, abort)) != 0; };
    uint32_t tc = 0, mc = 0, outs = 0, joins = 0;  // tiles; the warp's tiles and items with rows; joined items
    bool ok = true, more = walk.next(I);
    while (more) {
      const int g = I.g;
      const int shift = s && I.two ? I.toks0 : 0;  // the slot's first token within the item
      const int nrows = (s && I.two ? I.toks - I.toks0 : I.toks0) * g;
      const int pbase = I.p0 + shift;
      const int r0 = quarter * 32, rlast = min(r0 + 31, nrows - 1);
      const bool live = r0 < nrows;  // the warp holds rows
      auto token = [&](int r) { return PAGED ? r / g : r; };
      const int pos = pbase + token(row), wmin = pbase + token(r0), wmax = pbase + token(rlast);
      float m = kNegInf, l = 0.f;  // the reference of this thread's sum, and the sum
      bool any = false;            // a tile of this share is the slot's
      for (int j = I.next(0); j < I.T; j = I.next(j + 1)) {
        // what the step sees is found before its logits are waited for
        const int u0 = I.tile(j) * TILE + half * UNIT;
        const bool none = u0 > wmax || (u0 + UNIT - 1 <= wmin - p.window && u0 >= p.sinks);
        const bool whole = u0 + UNIT - 1 <= wmin && (u0 > wmax - p.window || u0 + UNIT <= p.sinks);
        const bool clear = PAGED && half == 0 &&
                           (u0 + TILE - 1 >= I.p0 + I.toks || (u0 <= I.p0 - p.window && u0 + TILE > p.sinks));
        if (!(ok = wait(&M.s_full[s][half], tc))) break;
        tc_fence_after();
        if (clear) clear_v(I, base + j, u0);
        if (live) {
          const uint32_t bad = PAGED ? (M.bad[(base + j) & 7] >> (half * 4)) & 15u : 0u;
          const bool all = whole && bad == 0;
          // 32 logits at a time stay in registers (96 a thread): the first half of them is read for its
          // maximum and once more for its weights.
          float x[32];
          auto load = [&](int q) {
            tmem_ld32(s_addr + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
            tmem_wait_ld();
            if (!all) {
              uint32_t vis = visible_keys(pos, u0 + 32 * q, p.window, p.sinks);
              if (PAGED) {
                const uint32_t gone = bad >> (2 * q);
                vis &= ~((gone & 1u ? 0xffffu : 0u) | (gone & 2u ? 0xffff0000u : 0u));
              }
#pragma unroll
              for (int c = 0; c < 32; ++c) x[c] = keep(vis, c, x[c], kNegInf);
            }
          };
          float a0 = kNegInf, a1 = kNegInf, a2 = kNegInf, a3 = kNegInf;
          if (!none) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              load(q);
#pragma unroll
              for (int c = 0; c < 32; c += 8) {
                a0 = max3(a0, x[c], x[c + 1]);
                a1 = max3(a1, x[c + 2], x[c + 3]);
                a2 = max3(a2, x[c + 4], x[c + 5]);
                a3 = max3(a3, x[c + 6], x[c + 7]);
              }
            }
          }
          const float mx = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)) * p.c;  // scale > 0
          // The maximum up to the step before: the other half's.
          float mp = kNegInf;
          if (half || any) {
            if (!(ok = wait(&M.m_ready[s][half ^ 1][quarter], mc - 1 + half))) break;
            mp = *mref;
          }
          // Raise it when the step exceeds it by more than the threshold; O (after the step before's P V)
          // is then rescaled.
          const bool need = mp != kNegInf && mx > mp + kRescaleThreshold;
          if (__any_sync(0xffffffffu, need)) {
            if (!(ok = wait(&M.pv_done[s][half ^ 1], tc - 1 + half))) break;
            tc_fence_after();
            const float f = need ? ex2(mp - mx) : 1.0f;
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 16) {
              uint32_t r[16];
              tmem_ld16(lane_base + HD * s + c0, r);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * f);
              tmem_st16(lane_base + HD * s + c0, r);
            }
          }
          const float mn = need || mp == kNegInf ? mx : mp;
          *mref = mn;
          __syncwarp();
          if (lane == 0) mbar_arrive(&M.m_ready[s][half][quarter]);
          ++mc;
          if (mn != m) {
            l *= ex2(m - mn);  // from -infinity by zero, which keeps a NaN
            m = mn;
          }
          const float nm = m == kNegInf ? 0.f : -m;
          uint32_t pk[16];
          if (none) {
#pragma unroll
            for (int c = 0; c < 16; ++c) pk[c] = 0u;
            tmem_st16(s_addr + 32, pk);
            tmem_st16(s_addr + 48, pk);
          } else {
            float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
            const float2 cc = make_float2(p.c, p.c), mm = make_float2(nm, nm);
#pragma unroll
            for (int q = 1; q >= 0; --q) {
              if (q == 0) load(0);
#pragma unroll
              for (int c = 0; c < 32; c += 4) {
                const float2 y0 = fma2(make_float2(x[c], x[c + 1]), cc, mm), y1 = fma2(make_float2(x[c + 2], x[c + 3]), cc, mm);
                const float2 e0 = make_float2(ex2(y0.x), ex2(y0.y)), e1 = make_float2(ex2(y1.x), ex2(y1.y));
                sum0 = add2(sum0, e0);
                sum1 = add2(sum1, e1);
                pk[c / 2] = pack_bf16(e0.x, e0.y);
                pk[c / 2 + 1] = pack_bf16(e1.x, e1.y);
              }
              tmem_st16(s_addr + 32 + 16 * q, pk);
            }
            l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M.p_full[s][half]);
        ++tc;
        any = true;
      }
      if (!ok) break;
      base += I.T;

      // ---- the row's statistics: the last published maximum, both halves' sums
      if (any && live) {
        if (half == 0) {
          if (!(ok = wait(&M.m_ready[s][1][quarter], mc - 1))) break;
          const float mn = *mref;
          if (mn != m) {
            l *= ex2(m - mn);  // from -infinity by zero, which keeps a NaN
            m = mn;
          }
          M.sum[s][row] = l;
          __syncwarp();
          if (lane == 0) mbar_arrive(&M.sum_ready[s][quarter]);
          if (!(ok = wait(&M.total_ready[s][quarter], outs))) break;
          l = M.sum[s][row];
        } else {
          if (!(ok = wait(&M.sum_ready[s][quarter], outs))) break;
          l += M.sum[s][row];
          M.sum[s][row] = l;
          __syncwarp();
          if (lane == 0) mbar_arrive(&M.total_ready[s][quarter]);
        }
        ++outs;
      }
      // ---- epilogue of the item: each half's warps take half of O's columns.  The next item's coordinates
      // (loads and divisions) are formed while the last product runs.
      Item J;
      more = walk.next(J);
      if (any) {
        if (!(ok = wait(&M.pv_done[s][1], tc - 1))) break;
        tc_fence_after();
      }
      const bool join = !I.two && I.T > 1;
      if (join && s == 1) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M.join_ready);
        if (!(ok = wait(&M.join_done, joins))) break;
      }
      if (I.two || s == 0) {
        float f0 = 1.f, f1 = 0.f;
        if (join) {
          if (!(ok = wait(&M.join_ready, joins))) break;
          tc_fence_after();
          const float m1 = live ? M.mref[1][row] : kNegInf, l1 = live ? M.sum[1][row] : 0.f, mm = fmaxf(m, m1);
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
          constexpr int W = HD / 2;
          const int tok = I.row0 + shift + token(row), head = I.head0 + (PAGED ? row % g : 0);
          float* po = nullptr;
          bf16* ho = nullptr;
          if (mine) {
            if (cut) {
              float* pb = p.part + (size_t)(2 * blockIdx.x + (I.seg ? 1 : 0)) * partial_floats(2 * TILE, HD);
              const int pr = shift * g + row;
              po = pb + (size_t)pr * HD + W * half;
              if (half == 0) {
                pb[2 * TILE * HD + pr] = m;
                pb[2 * TILE * HD + 2 * TILE + pr] = l;
              }
            } else {
              ho = row_ptr_w<bf16>(p.h, PAGED ? 0 : I.b, head, tok) + W * half;
              if (half == 0) {
                const int64_t o = PAGED ? (int64_t)head * p.batch.T + tok : ((int64_t)I.b * p.Hq + head) * p.N + tok;
                p.lse[o] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
              }
            }
          }
          const uint32_t o_addr = lane_base + HD * s + W * half;
          float2 z = make_float2(0.f, 0.f);
#pragma unroll 1
          for (int c0 = 0; c0 < W; c0 += 16) {
            uint32_t r[16];
            if (any) {
              tmem_ld16(o_addr + c0, r);
              tmem_wait_ld();
            }
            // a row without weight stays zero whatever the accumulator holds
#pragma unroll
            for (int c = 0; c < 16; ++c) r[c] = any && f0 != 0.f ? __float_as_uint(__uint_as_float(r[c]) * f0) : 0u;
            if (join) {
              uint32_t r1[16];
              tmem_ld16(o_addr + HD + c0, r1);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c)
                if (f1 != 0.f) r[c] = __float_as_uint(fmaf(__uint_as_float(r1[c]), f1, __uint_as_float(r[c])));
            }
#pragma unroll
            for (int c = 0; c < 16; c += 2)
              z = fma2(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), make_float2(0.f, 0.f), z);
            if (po != nullptr) {
#pragma unroll
              for (int c = 0; c < 16; c += 4)
                *reinterpret_cast<uint4*>(po + c0 + c) = make_uint4(r[c], r[c + 1], r[c + 2], r[c + 3]);
            } else if (ho != nullptr) {
              uint32_t h8[8];
#pragma unroll
              for (int c = 0; c < 8; ++c) h8[c] = pack_bf16(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1]));
              store_32b(ho + c0, h8, p.wide);
            }
          }
          if (z.x + z.y != 0.f && (po != nullptr || ho != nullptr)) M.again = 1;
        }
        if (join) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&M.join_done);
        }
      }
      if (join) ++joins;
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M.o_free[s]);
      }
      I = J;
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
  // every warp's rows and statistics are stored
  if (M.again && !M.abort) form_again<HD, PAGED>(p, M);
}

template <int HD, bool PAGED>
constexpr int smem_bytes() {
  return Cfg<HD, PAGED>::OFF_MISC + (int)sizeof(Misc);
}
static_assert(smem_bytes<128, true>() <= 232448, "shared memory of a CTA");

template <int HD, bool PAGED>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& vs, const TcParams& p,
                   int ctas, cudaStream_t st) {
  auto kern = win_fwd_tc_kernel<HD, PAGED>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<HD, PAGED>());
  if (e != cudaSuccess) return e;
  kern<<<ctas, NTHREADS, smem_bytes<HD, PAGED>(), st>>>(q, k, v, vs, p);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_win_fwd_tc(const WinDims& D, const WinFwdArgs& a, int32_t* status, cudaStream_t st) {
  CUtensorMap q, k, v, vs;
  TcParams p{};
  if (!win_tma_map(&q, a.q, D.B, D.Hq, D.N, TILE, D.d, &p.zq) || !win_tma_map(&k, a.k, D.B, D.Hkv, D.N, TILE, D.d, &p.zk) ||
      !win_tma_map(&v, a.v, D.B, D.Hkv, D.N, TILE, D.d, &p.zv) ||
      !win_tma_map(&vs, a.v, D.B, D.Hkv, D.sinks > 0 ? D.sinks : D.N, TILE, D.d, &p.zv))
    return cudaErrorInvalidValue;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
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
  p.wide = wide_rows(a.h);
  const int64_t planes = (int64_t)D.B * D.Hq;
  // Both slots share key tiles at 256 rows, take them in turn at 128: 167 us against 198 for 32 heads of 8192
  // tokens (window 1024, d = 128), 13.8 against 9.7 for 8 heads of 1021 (window 200, d = 64), where 256 leaves SMs idle.
  p.rows_item = planes * ((D.N + 255) / 256) >= kCtas ? 256 : 128;
  const int64_t items = planes * ((D.N + p.rows_item - 1) / p.rows_item);
  const int ctas = (int)(items < kCtas ? items : kCtas);
  return D.d == 64 ? launch<64, false>(q, k, v, vs, p, ctas, st) : launch<128, false>(q, k, v, vs, p, ctas, st);
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
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.h = a.h;
  p.lse = a.lse;
  p.status = status;
  p.Hq = D.Hq;
  p.g = D.g;
  p.window = D.window;
  p.sinks = D.sinks;
  p.c = D.scale * kLog2e;
  p.wide = wide_rows(a.h);
  p.table = a.table;
  p.page = D.page;
  p.num_pages = D.num_pages;
  p.max_pages = D.max_pages;
  p.batch = Batch{a.q_start, a.kv_len, D.seqs, D.T, D.max_pages * D.page, 2 * p.TQ, D.window, D.sinks, D.Hkv};
  p.part = static_cast<float*>(a.ws);
  cudaError_t e = D.d == 64 ? launch<64, true>(q, k, v, v, p, kCtas, st) : launch<128, true>(q, k, v, v, p, kCtas, st);
  if (e != cudaSuccess) return e;
  return launch_paged_join<TILE, 2 * TILE>(D, a, kCtas, 2 * p.TQ, st);
}

}  // namespace ssa
