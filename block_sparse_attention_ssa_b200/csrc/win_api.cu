// libssa C ABI: window attention with sinks and the paged cache (argument checks
// and dispatch; see include/ssa.h).
#include "nvtx_range.h"
#include "win_common.cuh"

namespace ssa {
namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxTokens = 1 << 24;
constexpr int kMaxPositions = 1 << 30;

bool scale_ok(float s) { return s > 0.f && s != __builtin_huge_valf(); }
bool aligned(const void* p, size_t n) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % n == 0; }

ssa_status_t check_window(const ssa_window_dims_t* in, WinDims* out, bool* empty) {
  if (in == nullptr) return SSA_ERR_INVALID_ARG;
  WinDims D{};
  D.B = in->B; D.Hq = in->Hq; D.Hkv = in->Hkv; D.N = in->N; D.d = in->d;
  D.window = in->window; D.sinks = in->sinks; D.scale = in->scale; D.dtype = in->dtype;
  if (D.B < 0 || D.Hq < 0 || D.N < 0 || D.Hkv < 1 || D.window < 1 || D.sinks < 0) return SSA_ERR_INVALID_ARG;
  if (D.dtype != SSA_F32 && D.dtype != SSA_BF16) return SSA_ERR_INVALID_ARG;
  if (!scale_ok(D.scale) || D.Hq % D.Hkv != 0) return SSA_ERR_INVALID_ARG;
  if ((D.d != 64 && D.d != 128) || D.N > kMaxTokens) return SSA_ERR_UNSUPPORTED;
  *empty = (int64_t)D.B * D.Hq == 0 || D.N == 0;
  // grid limits: planes in one grid dimension, tiles x planes in another
  if ((int64_t)D.B * D.Hq > 65535 || (int64_t)D.B * D.Hq * ((D.N + 63) / 64) > (1LL << 30)) return SSA_ERR_UNSUPPORTED;
  D.g = D.Hq / D.Hkv;
  if (D.window > D.N) D.window = D.N > 0 ? D.N : 1;
  if (D.sinks > D.N) D.sinks = D.N;
  *out = D;
  return SSA_OK;
}

ssa_status_t check_paged(const ssa_paged_dims_t* in, PagedDims* out, bool* empty) {
  if (in == nullptr) return SSA_ERR_INVALID_ARG;
  PagedDims D{};
  D.seqs = in->num_seqs; D.T = in->total_q; D.Hq = in->Hq; D.Hkv = in->Hkv; D.d = in->d; D.page = in->page;
  D.num_pages = in->num_pages; D.max_pages = in->max_pages; D.window = in->window; D.sinks = in->sinks;
  D.scale = in->scale; D.dtype = in->dtype;
  if (D.seqs < 0 || D.T < 0 || D.Hq < 0 || D.Hkv < 1 || D.num_pages < 1 || D.max_pages < 1 || D.window < 1 || D.sinks < 0)
    return SSA_ERR_INVALID_ARG;
  if (D.dtype != SSA_F32 && D.dtype != SSA_BF16) return SSA_ERR_INVALID_ARG;
  if (!scale_ok(D.scale) || D.Hq % D.Hkv != 0) return SSA_ERR_INVALID_ARG;
  if (D.d != 64 && D.d != 128) return SSA_ERR_UNSUPPORTED;
  if (D.page != 16 && D.page != 32 && D.page != 64 && D.page != 128 && D.page != 256) return SSA_ERR_UNSUPPORTED;
  D.g = D.Hq / D.Hkv;
  if (D.g > 64 || D.Hq > 65535 || D.T > kMaxPositions || D.seqs > kMaxPositions || (int64_t)D.max_pages * D.page > kMaxPositions)
    return SSA_ERR_UNSUPPORTED;
  *empty = D.seqs == 0 || D.T == 0 || D.Hq == 0;
  // positions stay below 2^30, so nothing lies behind a longer window or past more sinks
  if (D.window > kMaxPositions) D.window = kMaxPositions;
  if (D.sinks > kMaxPositions) D.sinks = kMaxPositions;
  *out = D;
  return SSA_OK;
}

// A [B, H, N, d] tensor as in the other entry points.  Inputs may broadcast batches and
// heads (stride 0), kRows inputs none; an output's rows and slices may not lie over one another.
enum Use { kInput, kRows, kOutput };

// Whether a tensor's rows are apart: by growing stride, each dimension steps over all that the ones before it span.
// (Layouts whose slices interleave without nesting are taken for meeting.)
bool apart(const int64_t (&st)[3], const int64_t (&n)[3], int d) {
  int by[3] = {0, 1, 2};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (st[by[j]] > st[by[j + 1]]) {
        const int x = by[j];
        by[j] = by[j + 1];
        by[j + 1] = x;
      }
  __int128 span = d;  // strides below 2^38, up to 2^31 slices
  for (int i : by) {
    if (n[i] <= 1) continue;
    if (st[i] < span) return false;
    span += (__int128)st[i] * (n[i] - 1);
  }
  return true;
}

ssa_status_t check_tensor(const ssa_tensor_t* t, int dtype, int d, int64_t B, int64_t H, int64_t N, Use use, TensorRef* out) {
  if (t == nullptr || !aligned(t->ptr, 16)) return SSA_ERR_INVALID_ARG;
  const int64_t es = dtype == SSA_BF16 ? 2 : 4;
  const int64_t st[3] = {t->stride_b, t->stride_h, t->stride_n}, n[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    if (st[i] < 0 || st[i] >= (1LL << 38) || (st[i] * es) % 16) return SSA_ERR_INVALID_ARG;
    // rows that overlap in part describe no tensor; slices laid over one another (stride 0) are a broadcast
    if (n[i] > 1 && st[i] < d && (use != kInput || i == 2 || st[i] != 0)) return SSA_ERR_INVALID_ARG;
  }
  if (use == kOutput && !apart(st, n, d)) return SSA_ERR_INVALID_ARG;
  *out = TensorRef{t->ptr, t->stride_b, t->stride_h, t->stride_n};
  return SSA_OK;
}

ssa_status_t check_ws(const void* ws, size_t have, size_t need) {
  if (ws == nullptr || have < need) return SSA_ERR_WORKSPACE;
  return aligned(ws, kAlign) ? SSA_OK : SSA_ERR_INVALID_ARG;
}

size_t paged_bytes(const PagedDims& D) { return D.dtype == SSA_F32 ? paged_ws_bytes(D) : paged_tc_ws_bytes(D); }

ssa_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? SSA_OK : SSA_ERR_CUDA; }

}  // namespace
}  // namespace ssa

using namespace ssa;

extern "C" {

size_t ssa_window_workspace_bytes(const ssa_window_dims_t* dims) {
  WinDims D;
  bool empty = false;
  if (check_window(dims, &D, &empty) != SSA_OK || empty) return 0;
  return win_bwd_layout(D).bytes;
}

ssa_status_t ssa_fwd_window(const ssa_window_dims_t* dims, const ssa_tensor_t* Q, const ssa_tensor_t* K,
                            const ssa_tensor_t* V, const ssa_tensor_t* h, float* lse, ssa_stream_t stream) {
  const NvtxRange nvtx_range("ssa_fwd_window");
  WinDims D;
  bool empty = false;
  ssa_status_t s = check_window(dims, &D, &empty);
  if (s != SSA_OK) return s;
  if (empty) return SSA_OK;
  WinFwdArgs a{};
  if ((s = check_tensor(Q, D.dtype, D.d, D.B, D.Hq, D.N, kInput, &a.q)) != SSA_OK) return s;
  if ((s = check_tensor(K, D.dtype, D.d, D.B, D.Hkv, D.N, kInput, &a.k)) != SSA_OK) return s;
  if ((s = check_tensor(V, D.dtype, D.d, D.B, D.Hkv, D.N, kInput, &a.v)) != SSA_OK) return s;
  if ((s = check_tensor(h, D.dtype, D.d, D.B, D.Hq, D.N, kOutput, &a.h)) != SSA_OK) return s;
  if (!aligned(lse, 4)) return SSA_ERR_INVALID_ARG;
  if ((s = require_sm100()) != SSA_OK) return s;
  a.lse = lse;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (D.dtype == SSA_F32) return from_cuda(launch_win_fwd_f32(D, a, st));
  int32_t* status = status_word();
  if (status == nullptr) return SSA_ERR_CUDA;
  return from_cuda(launch_win_fwd_tc(D, a, status, st));
}

ssa_status_t ssa_bwd_window(const ssa_window_dims_t* dims, const ssa_tensor_t* Q, const ssa_tensor_t* K,
                            const ssa_tensor_t* V, const ssa_tensor_t* h, const float* lse, const ssa_tensor_t* g,
                            const ssa_tensor_t* dQ, const ssa_tensor_t* dK, const ssa_tensor_t* dV, void* ws,
                            size_t ws_bytes, ssa_stream_t stream) {
  const NvtxRange nvtx_range("ssa_bwd_window");
  WinDims D;
  bool empty = false;
  ssa_status_t s = check_window(dims, &D, &empty);
  if (s != SSA_OK) return s;
  if (empty) return SSA_OK;
  WinBwdArgs a{};
  if ((s = check_tensor(Q, D.dtype, D.d, D.B, D.Hq, D.N, kInput, &a.q)) != SSA_OK) return s;
  if ((s = check_tensor(K, D.dtype, D.d, D.B, D.Hkv, D.N, kInput, &a.k)) != SSA_OK) return s;
  if ((s = check_tensor(V, D.dtype, D.d, D.B, D.Hkv, D.N, kInput, &a.v)) != SSA_OK) return s;
  if ((s = check_tensor(h, D.dtype, D.d, D.B, D.Hq, D.N, kInput, &a.h)) != SSA_OK) return s;
  if ((s = check_tensor(g, D.dtype, D.d, D.B, D.Hq, D.N, kInput, &a.g)) != SSA_OK) return s;
  if ((s = check_tensor(dQ, D.dtype, D.d, D.B, D.Hq, D.N, kOutput, &a.dq)) != SSA_OK) return s;
  if ((s = check_tensor(dK, D.dtype, D.d, D.B, D.Hkv, D.N, kOutput, &a.dk)) != SSA_OK) return s;
  if ((s = check_tensor(dV, D.dtype, D.d, D.B, D.Hkv, D.N, kOutput, &a.dv)) != SSA_OK) return s;
  if (!aligned(lse, 4)) return SSA_ERR_INVALID_ARG;
  if ((s = check_ws(ws, ws_bytes, win_bwd_layout(D).bytes)) != SSA_OK) return s;
  if ((s = require_sm100()) != SSA_OK) return s;
  a.lse = lse;
  a.ws = ws;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (D.dtype == SSA_F32) return from_cuda(launch_win_bwd_f32(D, a, st));
  int32_t* status = status_word();
  if (status == nullptr) return SSA_ERR_CUDA;
  return from_cuda(launch_win_bwd_tc(D, a, status, st));
}

size_t ssa_paged_workspace_bytes(const ssa_paged_dims_t* dims) {
  PagedDims D;
  bool empty = false;
  if (check_paged(dims, &D, &empty) != SSA_OK || empty) return 0;
  return paged_bytes(D);
}

ssa_status_t ssa_paged_append(const ssa_paged_dims_t* dims, const ssa_tensor_t* k, const ssa_tensor_t* v,
                              const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table,
                              const ssa_tensor_t* K, const ssa_tensor_t* V, ssa_stream_t stream) {
  const NvtxRange nvtx_range("ssa_paged_append");
  PagedDims D;
  bool empty = false;
  ssa_status_t s = check_paged(dims, &D, &empty);
  if (s != SSA_OK) return s;
  if (empty) return SSA_OK;
  PagedArgs a{};
  if ((s = check_tensor(k, D.dtype, D.d, 1, D.Hkv, D.T, kInput, &a.nk)) != SSA_OK) return s;
  if ((s = check_tensor(v, D.dtype, D.d, 1, D.Hkv, D.T, kInput, &a.nv)) != SSA_OK) return s;
  if ((s = check_tensor(K, D.dtype, D.d, D.num_pages, D.Hkv, D.page, kOutput, &a.k)) != SSA_OK) return s;
  if ((s = check_tensor(V, D.dtype, D.d, D.num_pages, D.Hkv, D.page, kOutput, &a.v)) != SSA_OK) return s;
  if (!aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4)) return SSA_ERR_INVALID_ARG;
  if ((s = require_sm100()) != SSA_OK) return s;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.table = page_table;
  return from_cuda(launch_paged_append(D, a, static_cast<cudaStream_t>(stream)));
}

ssa_status_t ssa_paged_attention(const ssa_paged_dims_t* dims, const ssa_tensor_t* q, const ssa_tensor_t* K,
                                 const ssa_tensor_t* V, const int32_t* q_start, const int32_t* kv_len,
                                 const int32_t* page_table, const ssa_tensor_t* h, float* lse, void* ws,
                                 size_t ws_bytes, ssa_stream_t stream) {
  const NvtxRange nvtx_range("ssa_paged_attention");
  PagedDims D;
  bool empty = false;
  ssa_status_t s = check_paged(dims, &D, &empty);
  if (s != SSA_OK) return s;
  if (empty) return SSA_OK;
  PagedArgs a{};
  // a slot's heads come in one TMA box: no broadcast of them
  if ((s = check_tensor(q, D.dtype, D.d, 1, D.Hq, D.T, kRows, &a.q)) != SSA_OK) return s;
  if ((s = check_tensor(K, D.dtype, D.d, D.num_pages, D.Hkv, D.page, kInput, &a.k)) != SSA_OK) return s;
  if ((s = check_tensor(V, D.dtype, D.d, D.num_pages, D.Hkv, D.page, kInput, &a.v)) != SSA_OK) return s;
  if ((s = check_tensor(h, D.dtype, D.d, 1, D.Hq, D.T, kOutput, &a.h)) != SSA_OK) return s;
  if (!aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4) || !aligned(lse, 4))
    return SSA_ERR_INVALID_ARG;
  if ((s = check_ws(ws, ws_bytes, paged_bytes(D))) != SSA_OK) return s;
  if ((s = require_sm100()) != SSA_OK) return s;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.table = page_table;
  a.lse = lse;
  a.ws = ws;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (D.dtype == SSA_F32) return from_cuda(launch_paged_f32(D, a, st));
  int32_t* status = status_word();
  if (status == nullptr) return SSA_ERR_CUDA;
  return from_cuda(launch_paged_tc(D, a, status, st));
}

}  // extern "C"
