// Eviction from the paged cache by accumulated attention weight: of a row with more entries than its
// budget the last `recent` stay and, per key head, of the others those with the largest weights (of
// equal ones the first); the kept entries move up in their order. The row's cache then has budget
// entries again ([R] "Speculative decoding", rayaq.ca ml-models -- Verification attention and the
// cache: what is not kept is dropped and the lengths shrink).
//
// One cluster of S CTAs per row and key head.
//   1  Selection. The order keys are read once into shared memory. Radix levels of up to 11 bits below the
//      keys' common prefix give the smallest kept key and how many of its equals stay; a bit per entry marks
//      the kept ones, with a running count per 128 entries. Every CTA does this on its own up to 16,384
//      entries. Of longer rows each takes a run, counts are added up over the cluster, and the CTAs copy each
//      other's bits.
//   2  Moves. Every CTA moves its share of the 16-byte columns of the entries' keys and values, in batches
//      of ascending destinations: all loads of a batch, a barrier, all its stores. A destination never
//      lies behind its source, so a batch's stores reach no entry that a later batch reads, and later
//      batches' loads need not wait. Columns are independent of each other: nothing else is waited for.
// Bound: the bytes of the moved entries, read and written once; entries before the first dropped one do
// not move. The cluster fills the GPU when rows and heads are few.
// Measured on fresh caches, with the launch, from a flushed L2 (D = 128, bf16, 8 heads): 32 rows of 2000 to 8190
// entries cut to 2048 101 us (5.2 TB/s), of which the selection takes 10; 3 rows of 1030 to 1501 cut to 1024
// 19 us; one row of 130,000 cut to 65,000 255 us, bound by the batches' round trips of 64 CTAs.
// A selection on the whole cluster for every length took 60 us of 8 us (two barriers of the cluster a level),
// one without it 600 us at 130,000 entries.

#include <climits>

#include "sv_cache.cuh"
#include "sv_common.cuh"

namespace {

constexpr int kInFlight = 8;               // 16-byte loads in flight per thread
constexpr int kMinCols = 2;                // columns of a CTA: at least a sector of an entry
constexpr int kBatchEach = 2;              // entries of a batch per thread, at most
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxRun = 1 << 18;           // entries of a run where rows are longest
constexpr size_t kSharedMost = 232448 - 512;   // of a CTA that has the SM alone
constexpr size_t kSharedOfTwo = 112 * 1024;   // dynamic shared memory of a CTA of which an SM holds two

struct EvictParams {
  sv::Cache C;
  const int32_t* length;
  int32_t* out_len;
  int budget, recent;
  int S;                                   // CTAs per row and head
  int words;                               // words of the kept bits, a multiple of 16
  int held;                                // order keys that shared memory holds
  int pages;                               // page numbers that it holds
};

// The weights' order: NaN above everything, -0 and 0 alike.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t x = w == 0.0f ? 0u : __float_as_uint(w);
  return (x & 0x80000000u) ? ~x : (x | 0x80000000u);
}

// Place of the set bit of v that has r others below it.
__device__ __forceinline__ int nth_bit(uint32_t v, int r) {
  int at = 0;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    const int c = __popc(v & ((1u << w) - 1u));
    if (r >= c) {
      r -= c;
      v >>= w;
      at += w;
    }
  }
  return at;
}

// What the CTAs of a cluster tell each other.
struct Told {
  uint32_t lo, hi;                         // range of the keys
  int bad, ties, kept, first;              // first: the first dropped entry
};

__device__ __forceinline__ uint32_t ld_cluster_u32(const void* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(sv::map_to_rank(sv::smem_addr(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_cluster_v2(const void* p, int rank) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y) : "r"(sv::map_to_rank(sv::smem_addr(p), rank)) : "memory");
  return v;
}
// The cluster's barrier, or the CTA's where it is alone.
__device__ __forceinline__ void meet(int S) {
  if (S > 1) sv::cluster_sync_all();
  else __syncthreads();
}

// Exclusive prefix sum over the CTA; *total gets the sum. tmp: one int per warp.
template <int kThreads>
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

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) sv_evict_kernel(const EvictParams P) {
  constexpr int kMaxBatch = kBatchEach * kThreads;
  extern __shared__ __align__(16) unsigned char dyn[];
  const sv::Cache& C = P.C;
  const int tid = threadIdx.x;
  const int rank = blockIdx.x % P.S, item = blockIdx.x / P.S;
  const int b = item / C.heads, h = item - b * C.heads;
  int* list = reinterpret_cast<int*>(dyn);                             // [2][kMaxBatch] sources
  uint32_t* bits = reinterpret_cast<uint32_t*>(list + 2 * kMaxBatch);  // kept entries
  int* before = reinterpret_cast<int*>(bits + P.words);                // kept before each 128 entries
  int* hist2 = before + P.words / 4;                                   // [2][kBins], levels in turn
  int* page_of = hist2 + 2 * kBins;                                    // [pages]
  uint32_t* keys = reinterpret_cast<uint32_t*>(page_of + P.pages);     // [held]
  __shared__ int tmp[kThreads / 32], sm_bin, sm_above, sm_count, sm_first;
  __shared__ uint32_t sm_lo[kThreads / 32], sm_hi[kThreads / 32];
  __shared__ Told mine;
  __shared__ int kept_of[kMaxCluster];     // kept entries before each run

  const int n = __ldg(P.length + b);
  const int S = n > P.held ? P.S : 1, part = n > P.held ? rank : 0;   // CTAs that share the selection
  const bool in_range = n >= 0 && n <= C.max_pages * C.page_size;
  const int old = n - P.recent, need = P.budget - P.recent;   // `need` of the first `old` entries stay
  const bool evicts = in_range && n > P.budget;
  const int32_t* table = C.table + static_cast<size_t>(b) * C.max_pages;
  const float* weights = C.weight + static_cast<size_t>(h) * C.page_size;
  const size_t page_floats = static_cast<size_t>(C.heads) * C.page_size;
  // This CTA's run: entries [e0, e1), whole blocks of 128.
  const int run = in_range ? ((n + S - 1) / S + 127) & ~127 : 0;
  const int e0 = min(part * run, max(n, 0)), e1 = min(e0 + run, max(n, 0));
  const bool held = e1 - e0 <= P.held;
  // Pages, and of a row that evicts the order keys of the run's old entries with their range.
  bool bad = !in_range;
  const int npages = in_range ? (n + C.page_size - 1) >> C.page_log2 : 0;
  const bool paged = npages <= P.pages;
  if (paged)
    for (int x = tid; x < npages; x += kThreads) page_of[x] = __ldg(table + x);
  auto page_at = [&](int j) { return paged ? page_of[j >> C.page_log2] : __ldg(table + (j >> C.page_log2)); };
  uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll 4
  for (int j = e0 + 4 * tid; j < e1; j += 4 * kThreads) {
    const int page = __ldg(table + (j >> C.page_log2));
    if (!sv::page_ok(C, page)) {
      bad = true;
      continue;
    }
    if (!evicts || need == 0 || j >= old) continue;
    const float4 w = *reinterpret_cast<const float4*>(weights + page * page_floats + (j & (C.page_size - 1)));
    const uint4 k = make_uint4(order_key(w.x), order_key(w.y), order_key(w.z), order_key(w.w));
    if (held) *reinterpret_cast<uint4*>(keys + j - e0) = k;
    const uint32_t e[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (j + x < old) {
        lo = min(lo, e[x]);
        hi = max(hi, e[x]);
      }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if ((tid & 31) == 0) {
    sm_lo[tid >> 5] = lo;
    sm_hi[tid >> 5] = hi;
  }
  bad = __syncthreads_or(bad);
  for (int x = 0; x < kThreads / 32; ++x) {
    lo = min(lo, sm_lo[x]);
    hi = max(hi, sm_hi[x]);
  }
  if (S > 1) {
    if (tid == 0) {
      mine.lo = lo;
      mine.hi = hi;
      mine.bad = bad;
    }
    meet(S);
    for (int r = 0; r < S; ++r) {
      lo = min(lo, ld_cluster_u32(&mine.lo, r));
      hi = max(hi, ld_cluster_u32(&mine.hi, r));
      bad |= ld_cluster_u32(&mine.bad, r) != 0;
    }
  }
  if (h == 0 && rank == 0 && tid == 0) P.out_len[b] = bad ? -1 : min(n, P.budget);
  if (bad || !evicts) {
    if (S > 1) meet(S);                      // the others have read what this one told
    return;                                  // the same for every CTA of the cluster
  }
  auto key_at = [&](int j) {
    return held ? keys[j - e0]
                : order_key(weights[__ldg(table + (j >> C.page_log2)) * page_floats + (j & (C.page_size - 1))]);
  };

  // 1. The smallest kept key, as `prefix` under `mask`: of the keys that equal it there `left` stay.
  uint32_t prefix = 0, mask = 0;
  int left = need;
  if (need > 0) {
    int bits_left = lo == hi ? 0 : 32 - __clz(lo ^ hi);
    mask = bits_left == 32 ? 0u : ~((1u << bits_left) - 1u);
    prefix = hi & mask;
    for (int level = 0; bits_left > 0; ++level) {
      const int nbits = min(bits_left, 11), shift = bits_left - nbits, nb = 1 << nbits;
      int* hist = hist2 + (level & 1) * kBins;
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int j = e0 + tid; j < min(e1, old); j += kThreads) {
        const uint32_t key = key_at(j);
        if ((key & mask) == prefix) atomicAdd(hist + (nb - 1 - ((key >> shift) & (nb - 1))), 1);   // largest first
      }
      meet(S);
      constexpr int kEach = kBins / kThreads;
      int c[kEach] = {};
      if (tid * kEach < nb) {
        if (S > 1)
          for (int r = 0; r < S; ++r)
#pragma unroll
            for (int x = 0; x < kEach; x += 2) {
              const uint2 v = ld_cluster_v2(hist + tid * kEach + x, r);
              c[x] += v.x;
              c[x + 1] += v.y;
            }
        else
#pragma unroll
          for (int x = 0; x < kEach; ++x) c[x] = hist[tid * kEach + x];
      }
      int sum = 0, total;
#pragma unroll
      for (int x = 0; x < kEach; ++x) sum += c[x];
      int at = block_excl_scan<kThreads>(sum, tmp, &total);
#pragma unroll
      for (int x = 0; x < kEach; ++x) {
        if (at < left && at + c[x] >= left) {      // one thread and bin
          sm_bin = nb - 1 - (tid * kEach + x);
          sm_above = at;
          sm_count = c[x];
        }
        at += c[x];
      }
      __syncthreads();
      left -= sm_above;
      prefix |= static_cast<uint32_t>(sm_bin) << shift;
      mask |= static_cast<uint32_t>(nb - 1) << shift;
      bits_left = sm_count == left ? 0 : shift;    // the whole bin stays: no need to look into it
      __syncthreads();
    }
  }
  // The kept bits of the run: keys above `prefix`, the first `left` entries that equal it, the recent ones.
  // A warp a word marks what is above and what is equal and counts the latter; with the count of the runs
  // before, a thread a word then keeps the first of them. The words of equals lie where the lists will be,
  // or where the keys would be if they were held.
  uint32_t* ties = held ? reinterpret_cast<uint32_t*>(list) : keys;
  const int nwords = (n + 31) >> 5, w0 = e0 >> 5, w1 = e1 > e0 ? (e1 + 31) >> 5 : w0;
  int count = 0;
#pragma unroll 4
  for (int w = w0 + (tid >> 5); w < w1; w += kThreads / 32) {
    const int j = 32 * w + (tid & 31);
    bool above = j < n && j >= old, tie = false;
    if (j < old && need > 0) {
      const uint32_t k = key_at(j) & mask;
      above = k > prefix;
      tie = k == prefix;
    }
    const uint32_t av = __ballot_sync(0xffffffffu, above), tv = __ballot_sync(0xffffffffu, tie);
    if ((tid & 31) == 0) {
      bits[w] = av;
      ties[w - w0] = tv;
      count += __popc(tv);
    }
  }
  int tie_run = 0, total;
  block_excl_scan<kThreads>(count, tmp, &total);
  if (S > 1) {
    if (tid == 0) mine.ties = total;
    meet(S);
    for (int r = 0; r < part; ++r) tie_run += static_cast<int>(ld_cluster_u32(&mine.ties, r));
  }
  if (tid == 0) {
    sm_first = INT_MAX;
    kept_of[0] = 0;
  }
  __syncthreads();
  int kept_run = 0;
  for (int x0 = w0; x0 < w1; x0 += kThreads) {
    const int w = x0 + tid;
    uint32_t keep = w < w1 ? bits[w] : 0u, tie = w < w1 ? ties[w - w0] : 0u;
    int t = tie_run + block_excl_scan<kThreads>(__popc(tie), tmp, &total);
    tie_run += total;
    while (tie && t < left) {
      keep |= tie & -tie;
      tie &= tie - 1;
      ++t;
    }
    const int k = kept_run + block_excl_scan<kThreads>(__popc(keep), tmp, &total);
    kept_run += total;
    if (w < w1) {
      bits[w] = keep;
      if ((w & 3) == 0) before[w >> 2] = k;
      const uint32_t full = 32 * w + 32 <= n ? 0xffffffffu : (1u << (n & 31)) - 1u;
      if (keep != full) atomicMin(&sm_first, 32 * w + __ffs(~keep & full) - 1);
    }
  }
  __syncthreads();
  int first = sm_first;
  if (S > 1) {
    // The other runs' bits and counts.
    if (tid == 0) {
      mine.kept = kept_run;
      mine.first = first;
    }
    meet(S);
    int sum = 0;
    for (int r = 0; r < S; ++r) {
      const int a = r * run >> 5, z = (min(r * run + run, n) + 31) >> 5;
      if (r != rank && r * run < n) {
        for (int w = a + tid; w < z; w += kThreads) bits[w] = ld_cluster_u32(bits + w, r);
        for (int w = (a >> 2) + tid; w < (z + 3) >> 2; w += kThreads)
          before[w] = static_cast<int>(ld_cluster_u32(before + w, r));
      }
      if (tid == 0) kept_of[r] = sum;
      sum += static_cast<int>(ld_cluster_u32(&mine.kept, r));
      first = min(first, static_cast<int>(ld_cluster_u32(&mine.first, r)));
    }
  }
  // Every CTA of the cluster has read the weights, and the others' bits, before any moves or leaves.
  meet(P.S);

  // 2. The moves, from the first dropped entry on.
  const int cols_log2 = (C.head_dim == 64 ? 4 : (C.head_dim == 128 ? 5 : 6)) - (31 - __clz(P.S));
  const int cols = 1 << cols_log2, vecs = C.head_dim / 8;
  const int per = kThreads >> cols_log2, batch = min(per * kInFlight, kMaxBatch);
  const int col = rank * cols + (tid & (cols - 1)), slot0 = tid >> cols_log2;
  char* base = (col < vecs ? C.k + col * 16 : C.v + (col - vecs) * 16);
  const int nblk = (nwords + 3) >> 2;
  auto build = [&](int d0, int* out) {       // the sources of destinations d0.. of a batch
    for (int x = tid; x < min(batch, P.budget - d0); x += kThreads) {
      const int d = d0 + x;
      int q = 0;                             // the run, then its last block with no more kept before it
      while (q + 1 < S && kept_of[q + 1] <= d) ++q;
      const int dq = d - kept_of[q];
      int lo = q * (run >> 7), hi = min(lo + (run >> 7), nblk);
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= dq) lo = mid;
        else hi = mid;
      }
      int r = dq - before[lo], wd = 4 * lo, c;
      while (r >= (c = __popc(bits[wd]))) {
        r -= c;
        ++wd;
      }
      out[x] = 32 * wd + nth_bit(bits[wd], r);
    }
  };
  int d0 = first;
  build(d0, list);
  __syncthreads();
  for (int cur = 0; d0 < P.budget; d0 += batch, cur ^= 1) {
    const int* L = list + cur * kMaxBatch;
    const int here = min(batch, P.budget - d0);
    uint4 x[kInFlight];
    float w[kBatchEach];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int e = u * per + slot0;
      if (e < here) x[u] = *reinterpret_cast<const uint4*>(base + sv::entry_offset(C, page_at(L[e]), h, L[e]));
    }
    if (rank == 0)                           // the weights are the first CTA's
#pragma unroll
      for (int y = 0; y < kBatchEach; ++y) {
        const int e = y * kThreads + tid;
        if (e < here) w[y] = *(C.weight + sv::weight_index(C, page_at(L[e]), h, L[e]));
      }
    build(d0 + batch, list + (cur ^ 1) * kMaxBatch);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int e = u * per + slot0;
      if (e < here) *reinterpret_cast<uint4*>(base + sv::entry_offset(C, page_at(d0 + e), h, d0 + e)) = x[u];
    }
    if (rank == 0)
#pragma unroll
      for (int y = 0; y < kBatchEach; ++y) {
        const int e = y * kThreads + tid;
        if (e < here) C.weight[sv::weight_index(C, page_at(d0 + e), h, d0 + e)] = w[y];
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
  const unsigned long long rows = 4ull * B;
  if (sv::overlap({{out_len, rows}}, {{length, rows}, sv::table_of(cache, B), sv::weights_of(cache),
                                      sv::pages_of(cache, cache->k), sv::pages_of(cache, cache->v)}))
    return SV_ERR_OVERLAP;
  int dev = 0;
  st = sv::current_device_status(&dev);
  if (st != SV_OK) return st;
  P.length = length;
  P.out_len = out_len;
  P.budget = budget;
  P.recent = recent;
  const long long items = static_cast<long long>(B) * P.C.heads;
  if (items > (1 << 27)) return SV_ERR_BAD_SHAPE;
  // Clusters as large as the SMs leave, or as the longest rows need. CTAs of 1024 threads, an SM each, where
  // that takes no threads away from the moves, else two of 512 an SM: a selection takes each CTA's threads
  // alone (16 rows of 5000 to 16,000 weights 33 us against 46, 8 of 130,000 255 against 326), but 64 rows and heads
  // of 9000 entries moved by 64 CTAs took 95 us, by 256 of half the size 67. A third of the SMs is left out: 16
  // clusters of 8 CTAs of 1024 threads did not run at once.
  // Lengths are on the device: what shared memory has to hold goes by the tables' room, and a table far wider than its
  // rows leaves less for keys and page numbers. 32 rows of 2000 to 8190 entries cut to 2048 take 111 us in tables that fit,
  // 137 in tables for 32,768 or 131,072 entries and 209 for 1,048,576; one row of 130,000 264 and, for 1,048,576, 450.
  const long long cap = static_cast<long long>(P.C.max_pages) * P.C.page_size;
  const int sms = sv::device_sms(dev);
  auto cluster = [&](long long most_ctas) {
    int S = 1;
    while (S < kMaxCluster && 2 * P.C.head_dim / 8 / (2 * S) >= kMinCols &&
           (2 * items * S <= most_ctas || cap > static_cast<long long>(kMaxRun) * S))
      S *= 2;
    return S;
  };
  const int large = cluster(2 * sms / 3), small = cluster(2 * sms);
  const bool alone = 3 * items <= 2 * sms && 2 * large >= small;
  P.S = alone ? large : small;
  P.words = static_cast<int>((cap / 32 + 15) / 16 * 16 + 16);
  // A half of an SM's shared memory, or all where a CTA has the SM alone: page numbers first,
  // then keys. Keys that are not held leave their place to a run's words of equals.
  const int threads = alone ? 1024 : 512;
  const size_t fixed = 2 * kBatchEach * threads * sizeof(int) + static_cast<size_t>(P.words) * 4 + P.words + 2 * kBins * sizeof(int);
  const long long all = alone ? kSharedMost : kSharedOfTwo, most_pages = alone ? 16384 : 4096;
  const long long most = cap < 16384 ? cap : 16384, least = cap > 16384 ? ((cap + P.S - 1) / P.S + 127) / 128 * 4 : 0;
  const long long ids = (P.C.max_pages + 3) / 4 * 4, fit = (static_cast<long long>(kSharedMost - fixed) - 4 * least) / 16 * 4;
  P.pages = static_cast<int>(ids < most_pages ? ids : most_pages);
  if (P.pages > fit) P.pages = static_cast<int>(fit);
  const long long room = (all - static_cast<long long>(fixed) - 4 * P.pages) / 16 * 4;
  P.held = static_cast<int>(room < least ? least : (room < most ? room : most));
  const size_t smem = fixed + 4 * static_cast<size_t>(P.pages) + static_cast<size_t>(P.held) * 4;
  static std::atomic<unsigned long long> allowed[2] = {};
  const auto kern = alone ? sv_evict_kernel<1024> : sv_evict_kernel<512>;
  if (sv::allow_shared(kern, kSharedMost, allowed[alone]) != SV_OK) return SV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * P.S));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(cuda_stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = P.S;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const EvictParams>(P)) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}
