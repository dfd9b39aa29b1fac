// What the kernels of the paged cache share: the cache as the device sees it, its entries' places,
// the two storage types, and the checks that every entry point makes on the host.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>

#include "../../include/spec_verify.h"

namespace sv {

// Entries a row of the cache may hold: the eviction keeps a bit for each and a count for each 128 of them in shared
// memory.
constexpr int kMaxEntries = 1 << 20;

struct Cache {
  char* k;
  char* v;
  float* weight;              // [num_pages, heads, page_size] or null
  const int32_t* table;       // [B, max_pages]
  long long page_stride, head_stride, slot_stride;   // bytes
  int num_pages, page_size, page_log2, max_pages, heads, head_dim;
};

__device__ __forceinline__ int cache_page(const Cache& C, int b, int j) {
  return __ldg(C.table + static_cast<size_t>(b) * C.max_pages + (j >> C.page_log2));
}
__device__ __forceinline__ bool page_ok(const Cache& C, int page) {
  return static_cast<unsigned>(page) < static_cast<unsigned>(C.num_pages);
}
// Byte offset of an entry's D elements in k or v.
__device__ __forceinline__ long long entry_offset(const Cache& C, int page, int h, int j) {
  return page * C.page_stride + h * C.head_stride + (j & (C.page_size - 1)) * C.slot_stride;
}
__device__ __forceinline__ size_t weight_index(const Cache& C, int page, int h, int j) {
  return (static_cast<size_t>(page) * C.heads + h) * C.page_size + (j & (C.page_size - 1));
}

// A row's entries before the round and its tokens; false when they are out of range. num: null means
// N; -1 (a row error of the verification) counts as no token where none_ok.
__device__ __forceinline__ bool round_lengths(const Cache& C, const int32_t* prefix,
                                              const int32_t* num, int b, int N, bool none_ok, int* n,
                                              int* m) {
  *n = __ldg(prefix + b);
  *m = num ? __ldg(num + b) : N;
  if (none_ok && *m == -1) *m = 0;
  if (*m < 0 || *m > N || *n < 0) return false;
  return static_cast<long long>(*n) + *m <= static_cast<long long>(C.max_pages) * C.page_size;
}

inline bool misaligned(const void* p, uintptr_t a) {
  return p && (reinterpret_cast<uintptr_t>(p) % a) != 0;
}

// An array of a call, from its first byte to its last (null: none).
struct Span {
  const void* p;
  unsigned long long bytes;
};
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && (x < y ? y - x < a.bytes : x - y < b.bytes);
}
// Whether one of the arrays that a call writes shares memory with another of them or with one that it reads.
inline bool overlap(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  for (const Span* w = written.begin(); w != written.end(); ++w) {
    for (const Span* x = w + 1; x != written.end(); ++x)
      if (overlap(*w, *x)) return true;
    for (const Span& r : read)
      if (overlap(*w, r)) return true;
  }
  return false;
}
// From the first element to the last of 16-bit elements, `inner` of them together, over three strided dimensions.
inline Span span_of(const void* p, int64_t inner, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2) {
  const __int128 e = static_cast<__int128>(n0 - 1) * s0 + static_cast<__int128>(n1 - 1) * s1 +
                     static_cast<__int128>(n2 - 1) * s2 + inner;
  const __int128 most = static_cast<__int128>(1) << 62;
  return {p, static_cast<unsigned long long>(2 * e < most ? 2 * e : most)};
}
// A cache's keys or values, its weights and its page table.
inline Span pages_of(const sv_paged_cache* c, const void* base) {
  return span_of(base, c->head_dim, c->num_pages, c->page_stride, c->heads, c->head_stride, c->page_size, c->slot_stride);
}
inline Span weights_of(const sv_paged_cache* c) {
  return {c->weight, 4ull * static_cast<unsigned>(c->num_pages) * static_cast<unsigned>(c->heads * c->page_size)};
}
inline Span table_of(const sv_paged_cache* c, int32_t B) {
  return {c->page_table, 4ull * static_cast<unsigned>(B) * static_cast<unsigned>(c->max_pages)};
}
// A round's [B, N, heads, D] input.
inline Span tokens_of(const void* x, int64_t row_stride, int64_t token_stride, int32_t B, int32_t N, int32_t heads, int32_t D) {
  return span_of(x, static_cast<int64_t>(heads) * D, B, row_stride, N, token_stride, 1, 0);
}

// The checks of a cache argument; fills the device form. need_weight: the call reads or writes weights.
inline int check_cache(const sv_paged_cache* c, int32_t B, bool need_weight, Cache* out) {
  if (!c || !c->k || !c->v || !c->page_table || (need_weight && !c->weight))
    return SV_ERR_NULL_POINTER;
  if (c->dtype != SV_DTYPE_BF16 && c->dtype != SV_DTYPE_F16) return SV_ERR_BAD_DTYPE;
  if (B < 1 || B > (1 << 20) || c->heads < 1 || c->heads > 1024 || c->num_pages < 1 ||
      c->max_pages < 1)
    return SV_ERR_BAD_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return SV_ERR_BAD_SHAPE;
  int lg = 4;
  while (lg < 8 && (1 << lg) != c->page_size) ++lg;
  if ((1 << lg) != c->page_size) return SV_ERR_BAD_SHAPE;
  if (static_cast<long long>(c->max_pages) * c->page_size > kMaxEntries) return SV_ERR_BAD_SHAPE;
  if (c->slot_stride < c->head_dim || (c->heads > 1 && c->head_stride < c->head_dim) ||
      (c->num_pages > 1 && c->page_stride < c->head_dim))
    return SV_ERR_BAD_SHAPE;
  const int64_t most = static_cast<int64_t>(1) << 38;      // a tensor map's strides stay below 2^40
  if (c->page_stride >= most || c->head_stride >= most || c->slot_stride >= most)
    return SV_ERR_BAD_SHAPE;
  if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->weight, 16) ||
      misaligned(c->page_table, 4) || c->page_stride % 8 != 0 || c->head_stride % 8 != 0 ||
      c->slot_stride % 8 != 0)
    return SV_ERR_MISALIGNED;
  out->k = static_cast<char*>(c->k);
  out->v = static_cast<char*>(c->v);
  out->weight = c->weight;
  out->table = c->page_table;
  out->page_stride = c->page_stride * 2;
  out->head_stride = c->head_stride * 2;
  out->slot_stride = c->slot_stride * 2;
  out->num_pages = c->num_pages;
  out->page_size = c->page_size;
  out->page_log2 = lg;
  out->max_pages = c->max_pages;
  out->heads = c->heads;
  out->head_dim = c->head_dim;
  return SV_OK;
}

// The checks of a round's [B, N, heads, D] input x (its strides in elements, its heads together).
inline int check_tokens(const void* x, int64_t row_stride, int64_t token_stride, int32_t B, int32_t N,
                        int32_t heads, int32_t D) {
  if (N < 1 || N > SV_MAX_GAMMA + 1 || heads < 1 || heads > 1024) return SV_ERR_BAD_SHAPE;
  const int64_t most = static_cast<int64_t>(1) << 38;
  if (row_stride < 0 || token_stride < 0 || row_stride >= most || token_stride >= most)
    return SV_ERR_BAD_SHAPE;
  if ((N > 1 && token_stride < static_cast<int64_t>(heads) * D) || (B > 1 && row_stride < heads * D))
    return SV_ERR_BAD_SHAPE;
  if (misaligned(x, 16) || row_stride % 8 != 0 || token_stride % 8 != 0) return SV_ERR_MISALIGNED;
  return SV_OK;
}

// A tensor map over the cache's keys or values (dimensions D, slot, head, page) whose boxes are 64
// elements (128 bytes, swizzled) of `rows` slots of one page and head.
int cache_tensor_map(const sv_paged_cache* c, const void* base, int rows, CUtensorMap* map);
// The same over a round's tokens (dimensions D, head, token, row): boxes of `heads` heads of `tokens` tokens.
int query_tensor_map(const void* q, int64_t row_stride, int64_t token_stride, int32_t B, int32_t N, int32_t Hq,
                     int32_t D, int32_t dtype, int heads, int tokens, CUtensorMap* map);
// Slots of one box: a page's, at most 64.
inline int box_rows(const sv_paged_cache* c) { return c->page_size < 64 ? c->page_size : 64; }
// Allows a kernel its dynamic shared memory on the current device, once (`done`: a bit per device).
template <typename K>
inline int allow_shared(K kern, size_t bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SV_ERR_CUDA;
  if ((done.load(std::memory_order_acquire) >> dev) & 1) return SV_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess)
    return SV_ERR_CUDA;
  done.fetch_or(1ull << dev, std::memory_order_release);
  return SV_OK;
}
// Multiprocessors of a device (sv_api.cu).
int device_sms(int dev);

// SV_OK when the current device is compute capability 10.3 (sv_api.cu).
int current_device_status(int* dev);

}  // namespace sv
