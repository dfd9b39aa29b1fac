// The attention weight that a round's kept tokens gave to each entry of the paged cache ([R]
// "Speculative decoding", rayaq.ca ml-models -- Verification attention and the cache):
//   weight_j += sum over kept tokens d with n_b + d >= j, and the key head's query heads, of
//               exp(scale q . k_j - lse).
//
// The simplest form: one CTA per row, key head and block of 64 entries; a warp takes every fourth entry
// of it and all its tokens, a lane D / 32 of the elements.

#include <cmath>

#include "sv_cache.cuh"
#include "sv_common.cuh"

namespace {

constexpr int kWarps = 4, kBlock = 64;

struct WeighParams {
  sv::Cache C;
  const char* q;
  long long row_stride, token_stride;   // bytes
  const float* lse;
  const int32_t* prefix;
  const int32_t* num;
  const int32_t* path;
  float c;                              // scale * log2(e)
  int N, Hq, group;
};

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) sv_weigh_plain_kernel(const WeighParams P) {
  const sv::Cache& C = P.C;
  const int h = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int E = D / 32;
  int n, m;
  bool bad = !sv::round_lengths(C, P.prefix, P.num, b, P.N, true, &n, &m);
  if (!bad && P.path && threadIdx.x < m) {
    const int i = __ldg(P.path + static_cast<size_t>(b) * P.N + threadIdx.x);
    bad = i < 0 || i >= P.N;
  }
  if (__syncthreads_or(bad)) return;
  for (int j0 = blockIdx.x * kBlock; j0 < n + m; j0 += gridDim.x * kBlock)
    for (int j = j0 + warp; j < min(j0 + kBlock, n + m); j += kWarps) {
      const int page = sv::cache_page(C, b, j);
      if (!sv::page_ok(C, page)) continue;
      const T* k = reinterpret_cast<const T*>(C.k + sv::entry_offset(C, page, h, j)) + lane * E;
      float kf[E];
#pragma unroll
      for (int e = 0; e < E; ++e) kf[e] = static_cast<float>(k[e]);
      float w = 0.0f;
      for (int d = max(0, j - n); d < m; ++d) {
        const int i = P.path ? __ldg(P.path + static_cast<size_t>(b) * P.N + d) : d;
        for (int g = 0; g < P.group; ++g) {
          const int hq = h * P.group + g;
          const T* q = reinterpret_cast<const T*>(P.q + b * P.row_stride + i * P.token_stride) + hq * D + lane * E;
          float s = 0.0f;
#pragma unroll
          for (int e = 0; e < E; ++e) s = fmaf(static_cast<float>(q[e]), kf[e], s);
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
          w += exp2f(s * P.c - __ldg(P.lse + (static_cast<size_t>(b) * P.N + i) * P.Hq + hq) * sv::kLog2e);
        }
      }
      if (lane == 0) atomicAdd(C.weight + sv::weight_index(C, page, h, j), w);
    }
}

}  // namespace

extern "C" int spec_verify_kv_weights(const void* q, int64_t q_row_stride, int64_t q_token_stride,
                                      const float* lse, const sv_paged_cache* cache,
                                      const int32_t* prefix_len, const int32_t* num_kept,
                                      const int32_t* path, float scale, int32_t B, int32_t N,
                                      int32_t Hq, void* cuda_stream) {
  WeighParams P;
  int st = sv::check_cache(cache, B, true, &P.C);
  if (st != SV_OK) return st;
  if (!q || !lse || !prefix_len) return SV_ERR_NULL_POINTER;
  st = sv::check_tokens(q, q_row_stride, q_token_stride, B, N, Hq, cache->head_dim);
  if (st != SV_OK) return st;
  if (Hq % cache->heads != 0 || !(scale > 0.0f) || !std::isfinite(scale)) return SV_ERR_BAD_SHAPE;
  if (sv::misaligned(lse, 4) || sv::misaligned(prefix_len, 4) || sv::misaligned(num_kept, 4) ||
      sv::misaligned(path, 4))
    return SV_ERR_MISALIGNED;
  int dev = 0;
  st = sv::current_device_status(&dev);
  if (st != SV_OK) return st;
  P.q = static_cast<const char*>(q);
  P.row_stride = q_row_stride * 2;
  P.token_stride = q_token_stride * 2;
  P.lse = lse;
  P.prefix = prefix_len;
  P.num = num_kept;
  P.path = path;
  P.c = scale * sv::kLog2e;
  P.N = N;
  P.Hq = Hq;
  P.group = Hq / cache->heads;
  const bool f16 = cache->dtype == SV_DTYPE_F16;
  void (*kern)(const WeighParams) = nullptr;
  switch (cache->head_dim) {
    case 64: kern = f16 ? sv_weigh_plain_kernel<__half, 64> : sv_weigh_plain_kernel<__nv_bfloat16, 64>; break;
    case 128: kern = f16 ? sv_weigh_plain_kernel<__half, 128> : sv_weigh_plain_kernel<__nv_bfloat16, 128>; break;
    default: kern = f16 ? sv_weigh_plain_kernel<__half, 256> : sv_weigh_plain_kernel<__nv_bfloat16, 256>; break;
  }
  const long long cap = static_cast<long long>(P.C.max_pages) * P.C.page_size;
  const int blocks = static_cast<int>((cap + kBlock - 1) / kBlock < 256 ? (cap + kBlock - 1) / kBlock : 256);
  kern<<<dim3(blocks, P.C.heads, B), 32 * kWarps, 0, static_cast<cudaStream_t>(cuda_stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
