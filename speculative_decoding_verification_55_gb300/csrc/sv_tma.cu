// Tensor maps of the paged cache for bulk tensor copies.

#include "sv_cache.cuh"

namespace {

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                             CUtensorMapFloatOOBfill);

EncodeFn find_encoder() {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult got = cudaDriverEntryPointSymbolNotFound;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &got) != cudaSuccess ||
      got != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<EncodeFn>(p);
}
// The driver's encoder, looked up once (a host function: the same for every device).
EncodeFn encode_fn() {
  static const EncodeFn fn = find_encoder();
  return fn;
}

}  // namespace

namespace sv {

namespace {

// A map of 16-bit elements over four dimensions (strides in elements; that of a dimension of one element is
// never used, so any valid value stands in for it) with swizzled boxes of 64 x box1 x box2.
int encode(const void* base, const int64_t (&dims)[4], const int64_t (&strides)[3], int32_t dtype, int box1,
           int box2, CUtensorMap* map) {
  const EncodeFn fn = encode_fn();
  if (!fn) return SV_ERR_CUDA;
  cuuint64_t d[4], st[3];
  for (int x = 0; x < 4; ++x) d[x] = static_cast<cuuint64_t>(dims[x]);
  for (int x = 0; x < 3; ++x) st[x] = static_cast<cuuint64_t>(dims[x + 1] > 1 ? strides[x] : dims[0]) * 2;
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2), 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  const CUtensorMapDataType t =
      dtype == SV_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return fn(map, t, 4, const_cast<void*>(base), d, st, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? SV_OK
             : SV_ERR_CUDA;
}

}  // namespace

int cache_tensor_map(const sv_paged_cache* c, const void* base, int rows, CUtensorMap* map) {
  return encode(base, {c->head_dim, c->page_size, c->heads, c->num_pages},
                {c->slot_stride, c->head_stride, c->page_stride}, c->dtype, rows, 1, map);
}

int query_tensor_map(const void* q, int64_t row_stride, int64_t token_stride, int32_t B, int32_t N, int32_t Hq,
                     int32_t D, int32_t dtype, int heads, int tokens, CUtensorMap* map) {
  return encode(q, {D, Hq, N, B}, {D, token_stride, row_stride}, dtype, heads, tokens, map);
}

}  // namespace sv
