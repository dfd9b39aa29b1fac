// Eviction from the paged cache by accumulated attention weight: of a row with more entries than its
// budget the last `recent` stay and, per key head, of the others those with the largest weights (of
// equal ones the first); the kept entries move up in their order. The row's cache then has budget
// entries again ([R] "Speculative decoding", rayaq.ca ml-models -- Verification attention and the
// cache: what is not kept is dropped and the lengths shrink).
//
// One cluster of S CTAs per row and key head. Every CTA
//   1  selects: three radix levels (11, 11 and 10 bits) over the weights' order keys give the smallest
//      kept key and how many of its equals stay; one more pass marks the kept entries in a bit per
//      entry, with a running count per 128 entries;
//   2  moves its share of the 16-byte columns of the entries' keys and values, in batches of ascending
//      destinations: all loads of a batch, a barrier, all its stores. A destination never lies behind
//      its source, so a batch's stores reach no entry that a later batch reads, and later batches' loads
//      need not wait. Columns are independent of each other: the CTAs of a cluster meet once, before the
//      first CTA's weights move.
// Bound: the bytes of the moved entries, read and written once; entries before the first dropped one do
// not move. Splitting columns over a cluster fills the GPU when rows and heads are few: the selection
// is then done S times, but it reads 4 bytes of an entry against its 4 D.

#include "sv_cache.cuh"
#include "sv_common.cuh"

namespace {

constexpr int kThreads = 512;
constexpr int kInFlight = 8;               // 16-byte loads in flight per thread
constexpr int kMinCols = 4;                // columns of a CTA: at least 64 bytes of an entry
constexpr int kMaxBatch = kInFlight * kThreads / kMinCols;
constexpr int kBins = 2048;

struct EvictParams {
  sv::Cache C;
  const int32_t* length;
  int32_t* out_len;
  int budget, recent;
  int S;                                   // CTAs per row and head
  int words;                               // words of the kept bits, a multiple of 4
};

// The weights' order: NaN above everything, -0 and 0 alike.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t x = w == 0.0f ? 0u : __float_as_uint(w);
  return (x & 0x80000000u) ? ~x : (x | 0x80000000u);
}

// Exclusive prefix sum over the CTA; *total gets the sum. tmp: one int per warp and one more.
__device__ __forceinline__ int block_excl_scan(int v, int* tmp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int t = lane < kThreads / 32 ? tmp[lane] : 0;
#pragma unroll
    for (int o = 1; o < kThreads / 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    if (lane < kThreads / 32) tmp[lane] = t;
  }
  __syncthreads();
  *total = tmp[kThreads / 32 - 1];
  const int before = warp ? tmp[warp - 1] : 0;
  __syncthreads();
  return before + x - v;
}

__global__ void __launch_bounds__(kThreads, 2) sv_evict_kernel(const EvictParams P) {
  extern __shared__ __align__(16) unsigned char dyn[];
  const sv::Cache& C = P.C;
  const int tid = threadIdx.x;
  const int rank = blockIdx.x % P.S, item = blockIdx.x / P.S;
  const int b = item / C.heads, h = item - b * C.heads;
  longlong2* list = reinterpret_cast<longlong2*>(dyn);                 // [2][kMaxBatch] from, to
  uint32_t* bits = reinterpret_cast<uint32_t*>(list + 2 * kMaxBatch);  // kept entries
  int* before = reinterpret_cast<int*>(bits + P.words);                // kept before each 128 entries
  int* hist = before + P.words / 4;
  __shared__ int tmp[kThreads / 32], sm_bin, sm_above, sm_first;

  const int n = __ldg(P.length + b);
  bool bad = n < 0 || n > C.max_pages * C.page_size;
  if (!bad)
    for (int p = tid; p < (n + C.page_size - 1) >> C.page_log2; p += kThreads)
      bad |= !sv::page_ok(C, __ldg(C.table + static_cast<size_t>(b) * C.max_pages + p));
  bad = __syncthreads_or(bad);
  if (h == 0 && rank == 0 && tid == 0) P.out_len[b] = bad ? -1 : min(n, P.budget);
  if (bad || n <= P.budget) return;          // the same for every CTA of the cluster

  // 1. The smallest kept key: `need` of the `old` entries stay.
  const int old = n - P.recent, need = P.budget - P.recent;
  uint32_t prefix = 0, mask = 0;
  int left = need;                           // still to find among the keys that match the prefix
  if (need > 0) {
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : (level == 1 ? 10 : 0), nb = level == 2 ? 1024 : 2048;
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int j = 4 * tid; j < old; j += 4 * kThreads) {
        const float4 w = *reinterpret_cast<const float4*>(
            C.weight + sv::weight_index(C, sv::cache_page(C, b, j), h, j));
        const float e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t key = order_key(e[x]);
          if (j + x < old && (key & mask) == prefix)
            atomicAdd(hist + (nb - 1 - ((key >> shift) & (nb - 1))), 1);   // largest keys first
        }
      }
      __syncthreads();
      int c[kBins / kThreads], sum = 0, total;
#pragma unroll
      for (int x = 0; x < kBins / kThreads; ++x) {
        c[x] = hist[tid * (kBins / kThreads) + x];
        sum += c[x];
      }
      int run = block_excl_scan(sum, tmp, &total);
#pragma unroll
      for (int x = 0; x < kBins / kThreads; ++x) {
        if (run < left && run + c[x] >= left) {    // one thread and bin
          sm_bin = nb - 1 - (tid * (kBins / kThreads) + x);
          sm_above = run;
        }
        run += c[x];
      }
      __syncthreads();
      left -= sm_above;
      prefix |= static_cast<uint32_t>(sm_bin) << shift;
      mask |= static_cast<uint32_t>(nb - 1) << shift;
      __syncthreads();
    }
  }
  // 2. The kept bits: keys above `prefix`, the first `left` entries that equal it, the recent ones.
  int kept_run = 0, tie_run = 0;
  if (tid == 0) sm_first = INT_MAX;
  __syncthreads();
  const int nwords = (n + 31) >> 5;
  for (int w0 = 0; w0 < ((nwords + 3) & ~3); w0 += kThreads) {
    const int w = w0 + tid;
    uint32_t above = 0, tie = 0;
    if (w < nwords) {
      for (int x = 0; x < 32; x += 4) {
        const int j = 32 * w + x;
        if (j >= n) break;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < old && need > 0)
          f = *reinterpret_cast<const float4*>(C.weight +
                                               sv::weight_index(C, sv::cache_page(C, b, j), h, j));
        const float e[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t key = order_key(e[y]), bit = 1u << (x + y);
          if (j + y >= n) continue;
          if (j + y >= old || (need > 0 && key > prefix)) above |= bit;
          else if (need > 0 && key == prefix) tie |= bit;
        }
      }
    }
    int total;
    int t = tie_run + block_excl_scan(__popc(tie), tmp, &total);
    tie_run += total;
    uint32_t keep = above;
    while (tie && t < left) {
      keep |= tie & -tie;
      tie &= tie - 1;
      ++t;
    }
    const int k = kept_run + block_excl_scan(__popc(keep), tmp, &total);
    kept_run += total;
    if (w < P.words) {
      bits[w] = keep;
      if ((w & 3) == 0) before[w >> 2] = k;
    }
    const uint32_t full = w < nwords ? (32 * w + 32 <= n ? 0xffffffffu : (1u << (n & 31)) - 1u) : 0u;
    if (keep != full) atomicMin(&sm_first, 32 * w + __ffs(~keep & full) - 1);
  }
  __syncthreads();
  // Every CTA of the cluster has read the weights before any of them moves.
  if (P.S > 1) sv::cluster_sync_all();

  // 3. The moves, from the first dropped entry on.
  const int cols_log2 = (C.head_dim == 64 ? 4 : (C.head_dim == 128 ? 5 : 6)) - (31 - __clz(P.S));
  const int cols = 1 << cols_log2, vecs = C.head_dim / 8;
  const int per = kThreads >> cols_log2, batch = per * kInFlight;
  const int col = rank * cols + (tid & (cols - 1)), slot0 = tid >> cols_log2;
  char* base = (col < vecs ? C.k + col * 16 : C.v + (col - vecs) * 16);
  const int nblk = (nwords + 3) >> 2;
  auto build = [&](int d0, longlong2* out, float (&w)[kMaxBatch / kThreads],
                   long long (&wto)[kMaxBatch / kThreads]) {
    // The places of destinations d0.. of a batch; CTA 0 also loads their weights.
#pragma unroll
    for (int y = 0; y < kMaxBatch / kThreads; ++y) {
      const int x = y * kThreads + tid, d = d0 + x;
      wto[y] = -1;
      if (x >= batch || d >= P.budget) continue;
      int lo = 0, hi = nblk;                 // the last block with before[] <= d
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= d) lo = mid;
        else hi = mid;
      }
      int r = d - before[lo], wd = 4 * lo, c;
      while (r >= (c = __popc(bits[wd]))) {
        r -= c;
        ++wd;
      }
      uint32_t v = bits[wd];
      for (; r > 0; --r) v &= v - 1;
      const int s = 32 * wd + __ffs(v) - 1;
      const int ps = sv::cache_page(C, b, s), pd = sv::cache_page(C, b, d);
      out[x] = make_longlong2(sv::entry_offset(C, ps, h, s), sv::entry_offset(C, pd, h, d));
      if (rank == 0) {
        w[y] = *reinterpret_cast<volatile const float*>(C.weight + sv::weight_index(C, ps, h, s));
        wto[y] = static_cast<long long>(sv::weight_index(C, pd, h, d));
      }
    }
  };
  float w[kMaxBatch / kThreads];
  long long wto[kMaxBatch / kThreads];
  int d0 = sm_first;
  build(d0, list, w, wto);
  __syncthreads();
  for (int cur = 0; d0 < P.budget; d0 += batch, cur ^= 1) {
    const longlong2* L = list + cur * kMaxBatch;
    uint4 x[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int e = u * per + slot0;
      if (d0 + e < P.budget) x[u] = *reinterpret_cast<const uint4*>(base + L[e].x);
    }
    float wn[kMaxBatch / kThreads];
    long long tn[kMaxBatch / kThreads];
    build(d0 + batch, list + (cur ^ 1) * kMaxBatch, wn, tn);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int e = u * per + slot0;
      if (d0 + e < P.budget) *reinterpret_cast<uint4*>(base + L[e].y) = x[u];
    }
#pragma unroll
    for (int y = 0; y < kMaxBatch / kThreads; ++y) {
      if (wto[y] >= 0) C.weight[wto[y]] = w[y];
      w[y] = wn[y];
      wto[y] = tn[y];
    }
    __syncthreads();
  }
}

}  // namespace

extern "C" int spec_verify_kv_evict(const sv_paged_cache* cache, const int32_t* length,
                                    int32_t budget, int32_t recent, int32_t* out_len, int32_t B,
                                    void* cuda_stream) {
  EvictParams P;
  int st = sv::check_cache(cache, B, true, &P.C);
  if (st != SV_OK) return st;
  if (!length || !out_len) return SV_ERR_NULL_POINTER;
  if (budget < 1 || recent < 0 || recent > budget) return SV_ERR_BAD_SHAPE;
  if (sv::misaligned(length, 4) || sv::misaligned(out_len, 4)) return SV_ERR_MISALIGNED;
  if (length == out_len) return SV_ERR_OVERLAP;
  int dev = 0;
  st = sv::current_device_status(&dev);
  if (st != SV_OK) return st;
  P.length = length;
  P.out_len = out_len;
  P.budget = budget;
  P.recent = recent;
  const long long items = static_cast<long long>(B) * P.C.heads;
  if (items > (1 << 27)) return SV_ERR_BAD_SHAPE;
  P.S = 1;
  while (P.S < 8 && items * P.S * 2 <= 304 && 2 * P.C.head_dim / 8 / (2 * P.S) >= kMinCols) P.S *= 2;
  const long long cap = static_cast<long long>(P.C.max_pages) * P.C.page_size;
  P.words = static_cast<int>((cap / 32 + 3) / 4 * 4 + 4);
  const size_t smem = 2 * kMaxBatch * sizeof(longlong2) + static_cast<size_t>(P.words) * 4 + P.words +
                      kBins * sizeof(int);
  if (cudaFuncSetAttribute(sv_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return SV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * P.S));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(cuda_stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = P.S;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sv_evict_kernel, static_cast<const EvictParams>(P)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}
