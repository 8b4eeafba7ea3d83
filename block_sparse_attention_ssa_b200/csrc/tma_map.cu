// TMA tensor maps over the [B, H, N, d] bf16 tensors of the tensor-core
// kernels (encoded on the host through the driver entry point, so that the
// library needs no libcuda at link time).
#include "ssa_internal.cuh"

#include <cudaTypedefs.h>

namespace ssa {

static PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (fn == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// 4-D map over a [B, H, N, d] bf16 tensor: dims (d, N, H, B), box (64, rows, 1, 1).
bool make_tma_map_bf16(CUtensorMap* map, const TensorRef& t, int B, int H, int N, int rows, int d) {
  auto enc = get_encode();
  if (enc == nullptr || (d != 64 && d != 128)) return false;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)H, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)t.sn * 2, (cuuint64_t)t.sh * 2, (cuuint64_t)t.sb * 2};
  // A zero stride (a broadcast dimension of size 1) is not accepted; any
  // positive multiple of 16 describes the same single slice.
  for (int i = 0; i < 3; ++i)
    if (strides[i] == 0) strides[i] = 16;
  cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(t.p), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 4-D bf16 map: dims (d, n1, n2, n3), strides of the outer three in elements, box (64, b1, b2, 1).
bool tma_map_4d(CUtensorMap* map, const void* p, int d, int64_t n1, int64_t n2, int64_t n3, int64_t s1, int64_t s2,
                int64_t s3, int b1, int b2) {
  auto enc = get_encode();
  if (enc == nullptr || (d != 64 && d != 128)) return false;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)n1, (cuuint64_t)n2, (cuuint64_t)n3};
  cuuint64_t strides[3] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2, (cuuint64_t)s3 * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)b1, (cuuint32_t)b2, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// A map takes no zero stride: a broadcast batch or head dimension gets one slice, and *zero says which
// coordinates stay 0 (bit 0 batch, bit 1 head).
bool win_tma_map(CUtensorMap* map, const TensorRef& t, int64_t B, int64_t H, int64_t N, int rows, int d, int* zero) {
  const bool zb = t.sb == 0 || B == 1, zh = t.sh == 0 || H == 1;
  *zero = (zb ? 1 : 0) | (zh ? 2 : 0);
  return tma_map_4d(map, t.p, d, N, zh ? 1 : H, zb ? 1 : B, N > 1 ? t.sn : 8, zh ? 8 : t.sh, zb ? 8 : t.sb, rows, 1);
}

bool fwd_tc_supported(const Dims& D) {
  return D.dtype == SSA_BF16 && D.d == 128 && (D.s == 64 || D.s == 128) && D.n <= 2048 && !D.per_token;
}

}  // namespace ssa
