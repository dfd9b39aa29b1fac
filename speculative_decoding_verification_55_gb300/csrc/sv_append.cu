// Append of a round's keys and values to the paged cache ([R] "Speculative decoding", rayaq.ca
// ml-models -- Verification attention and the cache: verification leaves an entry for each of the
// round's tokens; [B] brunomaga.github.io -- Medusa: of a tree only the kept path's entries stay).
//
// Bound: one read and one write of 4 D bytes per token and key head, small beside a launch for a decode
// step. A CTA has a group of a row's tokens (as many as leave six CTAs an SM, at most 16) and copies
// 16-byte columns, four loads in flight a thread; consecutive threads have consecutive columns of a token's
// keys, then of its values, so that reads and writes are whole lines. One token a CTA took 35 us for 512 rows
// of 31-node trees (84 MB moved), bound by the chain of loads that each CTA begins with; groups take 22.
// Every CTA of a row checks the whole row (its lengths, path and pages) before it writes anything: a
// row in error is left untouched.

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
  __shared__ int pages[SV_MAX_GAMMA + 1], from[SV_MAX_GAMMA + 1];
  const sv::Cache& C = P.C;
  const int b = blockIdx.x, tid = threadIdx.x;
  int n, m;
  bool ok = sv::round_lengths(C, P.prefix, P.num, b, P.N, true, &n, &m);
  if (ok) {
    bool bad = false;
    if (tid < m) {                       // m <= 65 tokens: one thread each
      const int i = P.path ? __ldg(P.path + static_cast<size_t>(b) * P.N + tid) : tid;
      const int page = sv::cache_page(C, b, n + tid);
      bad = !sv::page_ok(C, page) || i < 0 || i >= P.N;
      pages[tid] = page;
      from[tid] = i;
    }
    ok = !__syncthreads_or(bad);
  }
  if (blockIdx.y == 0 && tid == 0 && P.out_len) P.out_len[b] = ok ? n + m : -1;
  if (!ok) return;
  const int d0 = blockIdx.y * P.per, nd = min(P.per, m - d0);
  const int vec_log2 = C.head_dim == 64 ? 3 : (C.head_dim == 128 ? 4 : 5);   // 16-byte columns a head
  const int cols = C.heads << vec_log2;
  constexpr int kInFlight = 4;
  for (int x0 = tid; x0 < nd * 2 * cols; x0 += kInFlight * kAppendThreads) {
    uint4 e[kInFlight];
    char* to[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int x = x0 + u * kAppendThreads;
      to[u] = nullptr;
      if (x >= nd * 2 * cols) continue;
      const int d = d0 + x / (2 * cols), c = x % (2 * cols);
      const bool val = c >= cols;
      const int cc = val ? c - cols : c, h = cc >> vec_log2, at = cc & ((1 << vec_log2) - 1);
      e[u] = __ldg(reinterpret_cast<const uint4*>((val ? P.v_new : P.k_new) + b * P.row_stride +
                                                  from[d] * P.token_stride) + cc);
      to[u] = (val ? C.v : C.k) + sv::entry_offset(C, pages[d], h, n + d) + at * 16;
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (to[u]) *reinterpret_cast<uint4*>(to[u]) = e[u];
  }
  if (C.weight)
    for (int x = tid; x < nd * C.heads; x += kAppendThreads) {
      const int d = d0 + x / C.heads, h = x % C.heads;
      C.weight[sv::weight_index(C, pages[d], h, n + d)] = 0.0f;
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
  const unsigned long long rows = 4ull * B;
  const int32_t H = cache->heads, D = cache->head_dim;
  if (sv::overlap({{out_len, rows}},
                  {{prefix_len, rows}, {num_new, rows}, {path, rows * N}, sv::table_of(cache, B), sv::weights_of(cache),
                   sv::pages_of(cache, cache->k), sv::pages_of(cache, cache->v),
                   sv::tokens_of(k_new, row_stride, token_stride, B, N, H, D),
                   sv::tokens_of(v_new, row_stride, token_stride, B, N, H, D)}))
    return SV_ERR_OVERLAP;
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
  const long long sms = sv::device_sms(dev), each = static_cast<long long>(B) * N / (6 * (sms > 0 ? sms : 1));
  P.per = static_cast<int>(each < 1 ? 1 : (each > 16 ? 16 : each));
  sv_append_kernel<<<dim3(B, (N + P.per - 1) / P.per), kAppendThreads, 0,
                     static_cast<cudaStream_t>(cuda_stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
