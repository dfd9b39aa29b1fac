// Append of a round's keys and values to the paged cache ([R] "Speculative decoding", rayaq.ca
// ml-models -- Verification attention and the cache: verification leaves an entry for each of the
// round's tokens; [B] brunomaga.github.io -- Medusa: of a tree only the kept path's entries stay).
//
// Bound: one read and one write of 2 D elements per token and key head, small beside a launch. One CTA
// per row and group of tokens; consecutive threads copy consecutive 16-byte columns of a token's keys,
// then of its values, so that reads and writes are whole lines. Every CTA of a row checks the whole
// row (its lengths, path and pages) before it writes anything: a row in error is left untouched.

#include "sv_cache.cuh"

namespace {

constexpr int kAppendThreads = 256;

struct AppendParams {
  sv::Cache C;
  const char* k_new;
  const char* v_new;
  long long row_stride, token_stride;   // bytes
  const int32_t* prefix;
  const int32_t* num;
  const int32_t* path;
  int32_t* out_len;
  int N, per;                           // tokens of a row; tokens one CTA copies
};

__global__ void __launch_bounds__(kAppendThreads) sv_append_kernel(const AppendParams P) {
  const sv::Cache& C = P.C;
  const int b = blockIdx.x, tid = threadIdx.x;
  int n, m;
  bool ok = sv::round_lengths(C, P.prefix, P.num, b, P.N, true, &n, &m);
  if (ok) {
    bool bad = false;
    if (tid < m) {                       // m <= 65 tokens: one thread each
      bad = !sv::page_ok(C, sv::cache_page(C, b, n + tid));
      if (P.path) {
        const int i = __ldg(P.path + static_cast<size_t>(b) * P.N + tid);
        bad |= i < 0 || i >= P.N;
      }
    }
    ok = !__syncthreads_or(bad);
  }
  if (blockIdx.y == 0 && tid == 0 && P.out_len) P.out_len[b] = ok ? n + m : -1;
  if (!ok) return;
  const int d0 = blockIdx.y * P.per, d1 = min(d0 + P.per, m);
  const int vec_log2 = C.head_dim == 64 ? 3 : (C.head_dim == 128 ? 4 : 5);   // 16-byte columns a head
  const int cols = C.heads << vec_log2;
  for (int d = d0; d < d1; ++d) {
    const int i = P.path ? __ldg(P.path + static_cast<size_t>(b) * P.N + d) : d;
    const int j = n + d, page = sv::cache_page(C, b, j);
    const long long from = b * P.row_stride + i * P.token_stride;
    for (int c = tid; c < 2 * cols; c += kAppendThreads) {
      const bool val = c >= cols;
      const int cc = val ? c - cols : c, h = cc >> vec_log2, x = cc & ((1 << vec_log2) - 1);
      const uint4 e = __ldg(reinterpret_cast<const uint4*>((val ? P.v_new : P.k_new) + from) + cc);
      reinterpret_cast<uint4*>((val ? C.v : C.k) + sv::entry_offset(C, page, h, j))[x] = e;
    }
    if (C.weight)
      for (int h = tid; h < C.heads; h += kAppendThreads) C.weight[sv::weight_index(C, page, h, j)] = 0.0f;
  }
}

}  // namespace

extern "C" int spec_verify_kv_append(const void* k_new, const void* v_new, int64_t row_stride,
                                     int64_t token_stride, const sv_paged_cache* cache,
                                     const int32_t* prefix_len, const int32_t* num_new,
                                     const int32_t* path, int32_t* out_len, int32_t B, int32_t N,
                                     void* cuda_stream) {
  AppendParams P;
  int st = sv::check_cache(cache, B, false, &P.C);
  if (st != SV_OK) return st;
  if (!k_new || !v_new || !prefix_len) return SV_ERR_NULL_POINTER;
  st = sv::check_tokens(k_new, row_stride, token_stride, B, N, cache->heads, cache->head_dim);
  if (st != SV_OK) return st;
  if (sv::misaligned(v_new, 16) || sv::misaligned(prefix_len, 4) || sv::misaligned(num_new, 4) ||
      sv::misaligned(path, 4) || sv::misaligned(out_len, 4))
    return SV_ERR_MISALIGNED;
  if (out_len && (out_len == prefix_len || out_len == num_new || out_len == path)) return SV_ERR_OVERLAP;
  int dev = 0;
  st = sv::current_device_status(&dev);
  if (st != SV_OK) return st;
  P.k_new = static_cast<const char*>(k_new);
  P.v_new = static_cast<const char*>(v_new);
  P.row_stride = row_stride * 2;
  P.token_stride = token_stride * 2;
  P.prefix = prefix_len;
  P.num = num_new;
  P.path = path;
  P.out_len = out_len;
  P.N = N;
  P.per = 1;
  sv_append_kernel<<<dim3(B, (N + P.per - 1) / P.per), kAppendThreads, 0,
                     static_cast<cudaStream_t>(cuda_stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
