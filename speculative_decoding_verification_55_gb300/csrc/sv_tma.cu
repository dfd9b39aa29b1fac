// Tensor maps of the paged cache for bulk tensor copies.

#include <mutex>

#include "sv_cache.cuh"

namespace {

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                             CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (a host function: the same for every device).
EncodeFn encode_fn() {
  static std::once_flag once;
  static EncodeFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult got = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &got) == cudaSuccess &&
        got == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  });
  return fn;
}

}  // namespace

namespace sv {

int cache_tensor_map(const sv_paged_cache* c, const void* base, int rows, CUtensorMap* map) {
  const EncodeFn fn = encode_fn();
  if (!fn) return SV_ERR_CUDA;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->head_dim), static_cast<cuuint64_t>(c->page_size),
                              static_cast<cuuint64_t>(c->heads), static_cast<cuuint64_t>(c->num_pages)};
  // The stride of a dimension of one element is never used: any valid value stands in for it.
  const cuuint64_t strides[3] = {
      static_cast<cuuint64_t>(c->slot_stride) * 2,
      static_cast<cuuint64_t>(c->heads > 1 ? c->head_stride : c->slot_stride) * 2,
      static_cast<cuuint64_t>(c->num_pages > 1 ? c->page_stride : c->slot_stride) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  const CUtensorMapDataType t =
      c->dtype == SV_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return fn(map, t, 4, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? SV_OK
             : SV_ERR_CUDA;
}

}  // namespace sv
