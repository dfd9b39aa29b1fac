// The attention weight that a round's kept tokens gave to each entry of the paged cache ([R]
// "Speculative decoding", rayaq.ca ml-models -- Verification attention and the cache):
//   weight_j += sum over kept tokens d with n_b + d >= j, and the key head's query heads, of
//               exp(scale q . k_j - lse).
//
// One pass over the keys. The scores are S^T = K Q^T on the fifth-generation tensor cores: 128 entries
// are the rows and a key head's queries (tokens times heads, up to 128 at a time) the columns, so that
// a thread has one entry, adds up its row alone, and no thread needs another's numbers.
// Persistent CTAs take equal runs of the batch's key tiles (sv_tiles.cuh). Warps: one copies key tiles
// into a ring, one copies queries and tells the others what the item is, one thread issues the products
// into four buffers of tensor memory, and two groups of four take the tiles in turn. More than 128
// query rows go in chunks; more than two chunks' queries (one chunk's for heads of 256) are copied again for
// every tile (from L2). An entry's sum over its chunks stays with its thread, so that every entry gets a
// single addition.
// Bound: the bytes of the keys (32 KB a tile of 128 x 128 against 0.73 us of an SM's share of HBM; the
// products take 0.15 us at 72 rows, the exponentials 0.2).

#include <cmath>

#include "sv_tiles.cuh"
#include "sv_tmem.cuh"

namespace {

using namespace sv::tmem;
using sv::kFull;

constexpr int kTileLog2 = 7, kTile = 1 << kTileLog2;   // entries of a key tile
constexpr int kRows = 128;                             // query rows of a chunk
constexpr int kGroups = 2, kSoftWarps = 4 * kGroups, kSoft = 32 * kSoftWarps;
constexpr int kThreads = kSoft + 96;
constexpr int kProducer = kSoftWarps, kProducts = kSoftWarps + 1, kItems = kSoftWarps + 2;
constexpr int kOwn = 2, kScores = kOwn * kGroups;      // buffers of scores in tensor memory: of a group, all
constexpr int kPieces = 16;                            // items that the warps may be apart, and one
constexpr int kHeld = 8;                               // chunks whose rows' normalisers a group holds

struct WeighParams {
  sv::Round R;
  const float* lse;
  const int32_t* path;
  float c;                                             // scale * log2(e)
  int Hq, tokens;                                      // tokens of a chunk
};

template <int D>
constexpr int kSlotBytes = kTile * D * 2;
template <int D>
constexpr int kKeySlots = D == 64 ? 10 : (D == 128 ? 4 : 2);
template <int D>
constexpr int kQuerySlots = D == 256 ? 1 : 2;

struct Item {
  int row, head, first, count;                         // count 0: the end
  int n, m, bad;                                       // bad: a path entry out of range
};

template <int kK, int kQ>
struct Control {
  unsigned long long k_full[kK], k_empty[kK], q_full[kQ], q_empty[kQ], s_full[kScores], s_empty[kScores],
      told[kPieces], drained;
  long long scan[kThreads / 32];
  sv::Plan plan;
  Item items[kPieces];
  alignas(16) float nl[kGroups][kHeld][kRows];         // -lse log2(e) of an item's rows, by group and chunk
  int lost;
  uint32_t tm;
};
template <int D>
constexpr int kSmemBytes = (kKeySlots<D> + kQuerySlots<D>)*kSlotBytes<D> + sizeof(Control<kKeySlots<D>, kQuerySlots<D>>);

template <bool F16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    sv_weigh_kernel(const WeighParams P, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap qmap, int q_tokens) {
  constexpr int kK = kKeySlots<D>, kQ = kQuerySlots<D>;
  extern __shared__ __align__(1024) unsigned char dyn[];
  auto& S = *reinterpret_cast<Control<kK, kQ>*>(dyn + (kK + kQ) * kSlotBytes<D>);
  const sv::Round& R = P.R;
  const sv::Cache& C = R.C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = sv::smem_addr(dyn), qring = ring + kK * kSlotBytes<D>;
  if (tid == 0) {
    for (int s = 0; s < kK; ++s) {
      sv::mbar_init(sv::smem_addr(S.k_full + s), 1);
      sv::mbar_init(sv::smem_addr(S.k_empty + s), 1);
    }
    for (int s = 0; s < kQ; ++s) {
      sv::mbar_init(sv::smem_addr(S.q_full + s), 1);
      sv::mbar_init(sv::smem_addr(S.q_empty + s), 1);
    }
    for (int s = 0; s < kScores; ++s) {
      sv::mbar_init(sv::smem_addr(S.s_full + s), 1);
      sv::mbar_init(sv::smem_addr(S.s_empty + s), 4);
    }
    for (int s = 0; s < kPieces; ++s) sv::mbar_init(sv::smem_addr(S.told + s), 1);
    sv::mbar_init(sv::smem_addr(&S.drained), 1);
    S.lost = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kProducts) tm_alloc(&S.tm);
  sv::make_plan<kThreads>(R, S.scan, &S.plan);
  fence_after();
  const uint32_t tm = S.tm;
  volatile int* const lost = &S.lost;
  const int chunk_rows = P.tokens * R.group;
  // The next item's description. The items' warp always tells an end, however its own waits end: this wait is longer than
  // they can be, so that all warps know of the same items and meet at the same barriers.
  auto told = [&](int k) {
    Item I;
    if (sv::mbar_wait_drain(sv::smem_addr(S.told + k % kPieces), (k / kPieces) & 1)) I = S.items[k % kPieces];
    else {
      I.count = 0;
      *lost = 1;
    }
    return I;
  };
  // Chunks of an item; its queries are copied once when there is room for all, else for every tile.
  auto chunks_of = [&](const Item& I) { return (I.m + P.tokens - 1) / P.tokens; };

  if (warp == kProducer) {
    sv::Walk W;
    W.begin(R, S.plan);
    sv::TileLoader T;
    T.init(C, 1, kTileLog2);
    int armed = 0;
    bool gone = false;
    while (!gone && W.next(R)) {
      const int entries = W.w.n + W.w.m;
      const int last = W.first + W.count;
      const int32_t* const table = sv::pages_of(R, W.row, W.w);
      sv::PagesAhead pages;
      pages.begin(T, C, table, W.first, last, entries, lane);
      for (int t = W.first; t < last; ++t) {
        const int p = pages.next(T, C, table, t, last, entries, lane);
        const int s = armed % kK;
        const uint32_t bar = sv::smem_addr(S.k_full + s);
        if (armed >= kK &&
            !__all_sync(kFull, wait_unless_lost(sv::smem_addr(S.k_empty + s), (armed / kK - 1) & 1, lost))) {
          gone = true;
          break;
        }
        const int boxes = __popc(__ballot_sync(kFull, p >= 0));
        if (lane == 0) sv::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes) << (T.rows_log2 + 7));
        __syncwarp();
        if (p >= 0) T.load(C, &kmap, nullptr, t, W.head, p, lane, ring + s * kSlotBytes<D>, bar);
        ++armed;
      }
    }
    for (int e = max(0, armed - kK); e < armed; ++e)       // no copy is in flight when the CTA ends
      sv::mbar_wait_drain(sv::smem_addr(S.k_full + e % kK), (e / kK) & 1);
  } else if (warp == kProducts) {
    if (lane == 0) {
      // Places in the rings and buffers are counted on, not computed: this thread's own instructions take much
      // of a tile's time.
      const uint32_t k_full = sv::smem_addr(S.k_full), k_empty = sv::smem_addr(S.k_empty);
      const uint32_t q_full = sv::smem_addr(S.q_full), q_empty = sv::smem_addr(S.q_empty);
      const uint32_t s_full = sv::smem_addr(S.s_full), s_empty = sv::smem_addr(S.s_empty);
      const Matrix keys = matrix(ring, 16, 1024), queries = matrix(qring, 16, 1024);
      int ks = 0, g = 0, q = 0;                          // q: chunks of queries used up
      uint32_t k_phase = 0;
      // Score buffer of a group: `own` the next of its two, `turn` the phase that it is empty in.
      uint32_t own[kGroups] = {0, 0}, turn[kGroups] = {1, 1};
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const Item I = told(k);
        if (I.count == 0) break;
        const int chunks = chunks_of(I), rows = I.m * R.group;
        const bool stay = chunks <= kQ;
        for (int t = 0; t < I.count && ok; ++t) {
          ok = wait_unless_lost(k_full + 8 * ks, k_phase, lost);
          const Matrix km = keys.at(ks * kSlotBytes<D>);
          for (int x = 0; x < chunks && ok; ++x) {
            const uint32_t w = g * kOwn + (g ? own[1] : own[0]);
            // A buffer's first use finds it empty: waiting for the phase before its first returns at once.
            const int qx = stay ? q + x : q, qi = qx % kQ;
            ok = (stay && t > 0) || wait_unless_lost(q_full + 8 * qi, (qx / kQ) & 1, lost);
            ok = ok && wait_unless_lost(s_empty + 8 * w, g ? turn[1] : turn[0], lost);
            if (!ok) break;
            fence_after();
            const int n = (min(chunk_rows, rows - x * chunk_rows) + 15) & ~15;
            const uint32_t desc = product_desc<F16>(0, false) | (static_cast<uint32_t>(n >> 3) << 17);
            const Matrix qm = queries.at(qi * (kRows * D * 2));
#pragma unroll
            for (int y = 0; y < D / 16; ++y)
              product_ss(tm + w * kRows, km.at((y >> 2) * (kTile * 128) + (y & 3) * 32),
                         qm.at((y >> 2) * (kRows * 128) + (y & 3) * 32), desc, y > 0);
            products_done(s_full + 8 * w);
            if (x + 1 == chunks) products_done(k_empty + 8 * ks);
            if (!stay || t + 1 == I.count) products_done(q_empty + 8 * qi);   // this copy's last use
            if (!stay) ++q;
            if (g) {
              own[1] ^= 1u;
              if (own[1] == 0) turn[1] ^= 1u;
            } else {
              own[0] ^= 1u;
              if (own[0] == 0) turn[0] ^= 1u;
            }
          }
          if (++ks == kK) {
            ks = 0;
            k_phase ^= 1u;
          }
          g ^= 1;
        }
        if (stay) q += chunks;
      }
    }
    __syncwarp();
  } else if (warp == kItems) {
    sv::Walk W;
    W.begin(R, S.plan);
    int q = 0;
    for (int k = 0;; ++k) {
      const bool more = !__any_sync(kFull, *lost != 0) && W.next(R);
      bool bad = false;
      if (more && P.path)
        for (int d = lane; d < W.w.m; d += 32) {
          const int i = __ldg(P.path + static_cast<size_t>(W.row) * R.N + d);
          bad |= i < 0 || i >= R.N;
        }
      bad = __any_sync(kFull, bad);
      const Item I{W.row, W.head, W.first, more ? W.count : 0, W.w.n, W.w.m, bad ? 1 : 0};
      if (lane == 0) {
        S.items[k % kPieces] = I;
        sv::mbar_arrive(sv::smem_addr(S.told + k % kPieces));
      }
      if (!more) break;
      const int chunks = chunks_of(I);
      for (int x = 0; x < (chunks > kQ ? chunks * I.count : chunks); ++x, ++q) {
        const int qi = q % kQ;
        if (q >= kQ &&
            !__all_sync(kFull, wait_unless_lost(sv::smem_addr(S.q_empty + qi), (q / kQ - 1) & 1, lost)))
          break;                               // the next turn tells the end
        const int d0 = (x % chunks) * P.tokens;
        const uint32_t bar = sv::smem_addr(S.q_full + qi), to = qring + qi * (kRows * D * 2);
        // A chunk's tokens, q_tokens of them in a box; along a path, one by one.
        const int nt = P.path ? min(P.tokens, I.m - d0) : 1;
        if (lane == 0) sv::mbar_arrive_expect_tx(bar, (P.path ? nt : q_tokens) * R.group * D * 2);
        __syncwarp();
        for (int y = lane; y < nt * (D / 64); y += 32) {     // 64 elements of each head
          const int d = y / (D / 64), half = y % (D / 64);
          int i = d0 + d;
          if (P.path) i = min(max(__ldg(P.path + static_cast<size_t>(I.row) * R.N + i), 0), R.N - 1);
          sv::tma_load(to + half * (kRows * 128) + d * R.group * 128, &qmap, half * 64, I.head * R.group, i, I.row, bar);
        }
      }
    }
    for (int e = max(0, q - kQ); e < q; ++e)
      sv::mbar_wait_drain(sv::smem_addr(S.q_full + e % kQ), (e / kQ) & 1);
  } else {
    // ---- Sums: a thread an entry; the groups take the tiles in turn.
    const int g = warp >> 2, wq = warp & 3, wtid = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * wq) << 16;
    int tile = 0, unit = 0;
    bool ok = true;
    for (int k = 0;; ++k) {
      const Item I = told(k);
      if (I.count == 0) break;
      const int chunks = chunks_of(I), rows = I.m * R.group;
      bool loaded = false;                     // the item's normalisers are held
      for (int t = 0; t < I.count; ++t, ++tile) {
        if ((tile & 1) != g) continue;
        const int j = (I.first + t) * kTile + wtid;
        int page = -1;
        if (j < I.n + I.m) page = sv::cache_page(C, I.row, j);
        const bool mine = sv::page_ok(C, page) && !I.bad;
        float w = 0.0f;
        for (int x = 0; x < chunks; ++x, ++unit) {
          const int b = g * kOwn + unit % kOwn, r0 = x * chunk_rows, nr = min(chunk_rows, rows - r0);
          // All of an item's chunks at once, or kHeld of them at a time.
          if (!loaded || (chunks > kHeld && x % kHeld == 0)) {
            const int r1 = min(rows, r0 + kHeld * chunk_rows);
            sv::named_bar_sync(1 + g, 128);    // the group has read what was there
            for (int r = r0 + wtid; r < r1; r += 128) {
              const int d = r / R.group, hg = r - d * R.group, c = r / chunk_rows;
              int i = d;
              if (P.path) i = min(max(__ldg(P.path + static_cast<size_t>(I.row) * R.N + d), 0), R.N - 1);
              S.nl[g][c % kHeld][r - c * chunk_rows] =
                  -sv::kLog2e * __ldg(P.lse + (static_cast<size_t>(I.row) * R.N + i) * P.Hq + I.head * R.group + hg);
            }
            sv::named_bar_sync(1 + g, 128);
            loaded = true;
          }
          const float* const nl = S.nl[g][x % kHeld];
          ok = ok && __all_sync(kFull, wait_unless_lost(sv::smem_addr(S.s_full + b), (unit / kOwn) & 1, lost));
          if (!ok) continue;                   // a wait gave up: the barriers alone
          fence_after();
          // Rows before `lo` belong to tokens before the entry; rows from nr on are not there.
          const int lo = max(j - I.n, 0) * R.group - r0;
          const bool plain = __all_sync(kFull, lo <= 0);
          const sv::f32x2 c2 = sv::pk(P.c, P.c);
          sv::f32x2 sum[2] = {sv::pk(0.0f, 0.0f), sv::pk(0.0f, 0.0f)};
          for (int y = 0; y < nr; y += 32) {
            uint32_t s[32];
            tm_load32(s, tm + lanes + b * kRows + y);
            if (plain && y + 32 <= nr) {
#pragma unroll
              for (int z = 0; z < 32; z += 4) {
                const float4 e = *reinterpret_cast<const float4*>(nl + y + z);
                float p0, p1, p2, p3;
                sv::upk(sv::fma2(sv::pk(__uint_as_float(s[z]), __uint_as_float(s[z + 1])), c2, sv::pk(e.x, e.y)), p0, p1);
                sv::upk(sv::fma2(sv::pk(__uint_as_float(s[z + 2]), __uint_as_float(s[z + 3])), c2, sv::pk(e.z, e.w)), p2, p3);
                sum[0] = sv::add2(sum[0], sv::pk(sv::ex2(p0), sv::ex2(p1)));
                sum[1] = sv::add2(sum[1], sv::pk(sv::ex2(p2), sv::ex2(p3)));
              }
            } else {
              float a = 0.0f;
#pragma unroll
              for (int z = 0; z < 32; ++z) {
                const float p = sv::ex2(fmaf(__uint_as_float(s[z]), P.c, nl[y + z]));
                if (y + z >= lo && y + z < nr) a += p;
              }
              sum[0] = sv::add2(sum[0], sv::pk(a, 0.0f));
            }
          }
          float s0, s1;
          sv::upk(sv::add2(sum[0], sum[1]), s0, s1);
          w += s0 + s1;
          fence_before();
          __syncwarp();
          if (lane == 0) sv::mbar_arrive(sv::smem_addr(S.s_empty + b));
        }
        if (mine) atomicAdd(C.weight + sv::weight_index(C, page, I.head, j), w);
      }
    }
    fence_before();
  }
  __syncthreads();
  if (warp == kProducts) {
    if (S.lost && lane == 0) {                 // products in flight end before the tensor memory is given back
      products_done(sv::smem_addr(&S.drained));
      sv::mbar_wait_drain(sv::smem_addr(&S.drained), 0);
    }
    __syncwarp();
    tm_free(tm);
  }
  if (S.lost) {                                // a wait gave up: NaN for the whole run, whatever was added
    sv::Walk W;
    W.begin(R, S.plan);
    while (W.next(R)) {
      bool bad = false;                        // a row in error has no additions
      for (int d = 0; P.path && d < W.w.m; ++d) {
        const int i = __ldg(P.path + static_cast<size_t>(W.row) * R.N + d);
        bad |= i < 0 || i >= R.N;
      }
      const int stop = min((W.first + W.count) * kTile, W.w.n + W.w.m);
      for (int j = W.first * kTile + tid; j < stop && !bad; j += kThreads) {
        const int page = sv::cache_page(C, W.row, j);
        if (sv::page_ok(C, page))
          atomicAdd(C.weight + sv::weight_index(C, page, W.head, j), __int_as_float(0x7fffffff));
      }
    }
  }
}

template <bool F16, int D>
int launch(const WeighParams& P, const CUtensorMap& k, const CUtensorMap& q, int q_tokens, int grid, cudaStream_t st) {
  auto kern = sv_weigh_kernel<F16, D>;
  static std::atomic<unsigned long long> allowed{0};
  if (sv::allow_shared(kern, (kSmemBytes<D>), allowed) != SV_OK) return SV_ERR_CUDA;
  kern<<<grid, kThreads, kSmemBytes<D>, st>>>(P, k, q, q_tokens);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace

extern "C" int spec_verify_kv_weights(const void* q, int64_t q_row_stride, int64_t q_token_stride,
                                      const float* lse, const sv_paged_cache* cache,
                                      const int32_t* prefix_len, const int32_t* num_kept,
                                      const int32_t* path, float scale, int32_t B, int32_t N,
                                      int32_t Hq, void* cuda_stream) {
  WeighParams P;
  int st = sv::check_cache(cache, B, true, &P.R.C);
  if (st != SV_OK) return st;
  if (!q || !lse || !prefix_len) return SV_ERR_NULL_POINTER;
  st = sv::check_tokens(q, q_row_stride, q_token_stride, B, N, Hq, cache->head_dim);
  if (st != SV_OK) return st;
  if (Hq % cache->heads != 0 || Hq / cache->heads > kRows || !(scale > 0.0f) || !std::isfinite(scale))
    return SV_ERR_BAD_SHAPE;
  if (sv::misaligned(lse, 4) || sv::misaligned(prefix_len, 4) || sv::misaligned(num_kept, 4) ||
      sv::misaligned(path, 4))
    return SV_ERR_MISALIGNED;
  const unsigned long long row_bytes = 4ull * B;
  if (sv::overlap({sv::weights_of(cache)},
                  {sv::tokens_of(q, q_row_stride, q_token_stride, B, N, Hq, cache->head_dim), {lse, row_bytes * N * Hq},
                   {prefix_len, row_bytes}, {num_kept, row_bytes}, {path, row_bytes * N}, sv::table_of(cache, B),
                   sv::pages_of(cache, cache->k), sv::pages_of(cache, cache->v)}))
    return SV_ERR_OVERLAP;
  int dev = 0;
  st = sv::current_device_status(&dev);
  if (st != SV_OK) return st;
  const int D = cache->head_dim, group = Hq / cache->heads;
  const int chunk = kRows / group, tokens = path ? 1 : (chunk < N ? chunk : N);
  CUtensorMap kmap, qmap;
  st = sv::cache_tensor_map(cache, cache->k, sv::box_rows(cache), &kmap);
  if (st == SV_OK) st = sv::query_tensor_map(q, q_row_stride, q_token_stride, B, N, Hq, D, cache->dtype, group, tokens, &qmap);
  if (st != SV_OK) return st;
  P.R.prefix = prefix_len;
  P.R.num = num_kept;
  P.R.B = B;
  P.R.N = N;
  P.R.group = group;
  P.R.q_rows = N * group;                  // one item per row and key head
  P.R.tile_log2 = kTileLog2;
  P.R.extra = 2;
  P.R.none_ok = true;
  P.lse = lse;
  P.path = path;
  P.c = scale * sv::kLog2e;
  P.Hq = Hq;
  P.tokens = chunk;
  const int sms = sv::device_sms(dev);
  if (sms < 1) return SV_ERR_CUDA;
  const long long most = static_cast<long long>(B) * cache->heads *
                         ((static_cast<long long>(cache->max_pages) * cache->page_size + kTile - 1) / kTile);
  const int grid = static_cast<int>(most < sms ? most : sms);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool f16 = cache->dtype == SV_DTYPE_F16;
  if (D == 64) return f16 ? launch<true, 64>(P, kmap, qmap, tokens, grid, s) : launch<false, 64>(P, kmap, qmap, tokens, grid, s);
  if (D == 128) return f16 ? launch<true, 128>(P, kmap, qmap, tokens, grid, s) : launch<false, 128>(P, kmap, qmap, tokens, grid, s);
  return f16 ? launch<true, 256>(P, kmap, qmap, tokens, grid, s) : launch<false, 256>(P, kmap, qmap, tokens, grid, s);
}
