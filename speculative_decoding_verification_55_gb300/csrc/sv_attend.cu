// Attention of a round's tokens over the paged cache ([R] "Speculative decoding", rayaq.ca ml-models
// -- Verification attention and the cache; [B] brunomaga.github.io -- Medusa, tree attention).
//
//   s_ij = scale q_i . k_j,  out_i = sum_j p_ij v_j,  p_ij = exp(s_ij - lse_i),  over the entries j < n_b
//   of row b, token i itself, and the round's tokens before it (a chain) or above it (a tree).
//
// The simplest form: one CTA per row, token and query head; its warps take every fourth entry, a lane
// D / 32 of its elements, with a running maximum and sum each, joined at the end.

#include <cmath>

#include "sv_cache.cuh"
#include "sv_common.cuh"

namespace {

constexpr int kWarps = 4;

struct AttendParams {
  sv::Cache C;
  const char* q;
  long long row_stride, token_stride;   // bytes
  const int32_t* prefix;
  const int32_t* num;
  const int32_t* parents;
  void* out;
  float* lse;
  float c;                              // scale * log2(e)
  int N, Hq, group;
};

template <typename T>
__device__ __forceinline__ float to_f(T x) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) return __half2float(x);
  else return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T from_f(float x) {
  if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) sv_attend_plain_kernel(const AttendParams P) {
  const sv::Cache& C = P.C;
  const int hq = blockIdx.x, i = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int E = D / 32;
  __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][D];
  __shared__ int sm_bad;
  int n, m;
  bool ok = sv::round_lengths(C, P.prefix, P.num, b, P.N, false, &n, &m);
  T* out = static_cast<T*>(P.out) + ((static_cast<size_t>(b) * P.N + i) * P.Hq + hq) * D;
  float* lse = P.lse ? P.lse + (static_cast<size_t>(b) * P.N + i) * P.Hq + hq : nullptr;
  if (!ok || i >= m) {
    const float v = ok ? 0.0f : __int_as_float(0x7fc00000);
    for (int d = threadIdx.x; d < D; d += blockDim.x) out[d] = from_f<T>(v);
    if (threadIdx.x == 0 && lse) *lse = v;
    return;
  }
  if (threadIdx.x == 0) sm_bad = 0;
  // Ancestors of token i and the validity of the row's tree.
  const int32_t* par = P.parents ? P.parents + static_cast<size_t>(b) * P.N : nullptr;
  bool bad = false;
  if (par)
    for (int t = threadIdx.x; t < m; t += blockDim.x) {
      const int p = __ldg(par + t);
      bad |= t == 0 ? p != -1 : (p < 0 || p >= t);
    }
  bad = __syncthreads_or(bad);
  unsigned long long seen = 0;          // tokens 1..64 that token i attends, as bits 0..63
  if (par && !bad)
    for (int t = i; t > 0; t = __ldg(par + t)) seen |= 1ull << (t - 1);
  const int h = hq / P.group;
  const T* q = reinterpret_cast<const T*>(P.q + b * P.row_stride + i * P.token_stride) + hq * D;
  float qf[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qf[e] = to_f<T>(q[lane * E + e]);
    o[e] = 0.0f;
  }
  float mx = -INFINITY, l = 0.0f;
  if (!bad)
    for (int j = warp; j < n + m; j += kWarps) {
      if (j >= n) {
        const int t = j - n;
        if (par ? (t > 0 && !((seen >> (t - 1)) & 1)) : t > i) continue;
      }
      const int page = sv::cache_page(C, b, j);
      if (!sv::page_ok(C, page)) {
        bad = true;
        break;
      }
      const long long at = sv::entry_offset(C, page, h, j);
      const T* k = reinterpret_cast<const T*>(C.k + at);
      const T* v = reinterpret_cast<const T*>(C.v + at);
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(qf[e], to_f<T>(k[lane * E + e]), s);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      s *= P.c;
      const float nm = fmaxf(mx, s);
      const float f = mx == nm ? 1.0f : exp2f(mx - nm);
      const float p = s == -INFINITY ? 0.0f : exp2f(s - nm);
      l = l * f + p;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * to_f<T>(v[lane * E + e]);
      mx = nm;
    }
  if (bad) sm_bad = 1;
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = o[e];
  if (lane == 0) {
    sm_m[warp] = mx;
    sm_l[warp] = l;
  }
  __syncthreads();
  float M = -INFINITY, L = 0.0f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w]);
  float f[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    f[w] = sm_m[w] == -INFINITY ? 0.0f : exp2f(sm_m[w] - M);
    L += sm_l[w] * f[w];
  }
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float x = 0.0f;
    for (int w = 0; w < kWarps; ++w)
      if (f[w] != 0.0f) x += sm_o[w][d] * f[w];
    out[d] = from_f<T>(sm_bad ? __int_as_float(0x7fc00000) : x / L);
  }
  if (threadIdx.x == 0 && lse)
    *lse = sm_bad ? __int_as_float(0x7fc00000) : (M + log2f(L)) * 0.6931471805599453f;
}

}  // namespace

extern "C" size_t spec_verify_paged_attention_workspace_size(int32_t N, int32_t Hq,
                                                             const sv_paged_cache* cache) {
  if (!cache || N < 1 || N > SV_MAX_GAMMA + 1 || Hq < 1 || Hq > 1024 || cache->heads < 1 ||
      Hq % cache->heads != 0)
    return 0;
  return SV_ATTEND_COUNTER_BYTES;
}

extern "C" int spec_verify_paged_attention(const void* q, int64_t q_row_stride,
                                           int64_t q_token_stride, const sv_paged_cache* cache,
                                           const int32_t* prefix_len, const int32_t* num_queries,
                                           const int32_t* tree_parents, float scale, void* out,
                                           float* out_lse, int32_t B, int32_t N, int32_t Hq,
                                           void* workspace, size_t workspace_bytes,
                                           void* cuda_stream) {
  AttendParams P;
  int st = sv::check_cache(cache, B, false, &P.C);
  if (st != SV_OK) return st;
  if (!q || !prefix_len || !out) return SV_ERR_NULL_POINTER;
  st = sv::check_tokens(q, q_row_stride, q_token_stride, B, N, Hq, cache->head_dim);
  if (st != SV_OK) return st;
  if (Hq % cache->heads != 0 || !(scale > 0.0f) || !std::isfinite(scale)) return SV_ERR_BAD_SHAPE;
  if (sv::misaligned(out, 16) || sv::misaligned(out_lse, 4) || sv::misaligned(prefix_len, 4) ||
      sv::misaligned(num_queries, 4) || sv::misaligned(tree_parents, 4) ||
      sv::misaligned(workspace, 256))
    return SV_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < spec_verify_paged_attention_workspace_size(N, Hq, cache))
    return SV_ERR_WORKSPACE_TOO_SMALL;
  int dev = 0;
  st = sv::current_device_status(&dev);
  if (st != SV_OK) return st;
  P.q = static_cast<const char*>(q);
  P.row_stride = q_row_stride * 2;
  P.token_stride = q_token_stride * 2;
  P.prefix = prefix_len;
  P.num = num_queries;
  P.parents = tree_parents;
  P.out = out;
  P.lse = out_lse;
  P.c = scale * sv::kLog2e;
  P.N = N;
  P.Hq = Hq;
  P.group = Hq / cache->heads;
  const bool f16 = cache->dtype == SV_DTYPE_F16;
  void (*kern)(const AttendParams) = nullptr;
  switch (cache->head_dim) {
    case 64: kern = f16 ? sv_attend_plain_kernel<__half, 64> : sv_attend_plain_kernel<__nv_bfloat16, 64>; break;
    case 128: kern = f16 ? sv_attend_plain_kernel<__half, 128> : sv_attend_plain_kernel<__nv_bfloat16, 128>; break;
    default: kern = f16 ? sv_attend_plain_kernel<__half, 256> : sv_attend_plain_kernel<__nv_bfloat16, 256>; break;
  }
  kern<<<dim3(Hq, N, B), 32 * kWarps, 0, static_cast<cudaStream_t>(cuda_stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
