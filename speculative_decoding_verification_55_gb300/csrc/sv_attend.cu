// Attention of a round's tokens over the paged cache ([R] "Speculative decoding", rayaq.ca ml-models
// -- Verification attention and the cache; [B] brunomaga.github.io -- Medusa, tree attention).
//
//   s_ij = scale q_i . k_j,  out_i = sum_j p_ij v_j,  p_ij = exp(s_ij - lse_i),  over the entries j < n_b
//   of row b, token i itself, and the round's tokens before it (a chain) or above it (a tree).
//
// One pass over keys and values with a running maximum and sum per query row. The query rows of a key
// head (its query heads times the row's tokens) are the rows of the matrix products, so grouped heads
// and a round's tokens share every key and value that is read. Persistent CTAs take equal runs of the
// batch's key tiles (sv_tiles.cuh); an item that several CTAs share is joined from partial sums in the
// workspace (sv_attend_join.cu). This file holds the kernel for up to 16 query rows a key head, the others
// are in sv_attend_wide.cu.
//
// A CTA is one producer warp, which copies key tiles from the pages into a ring, and four consumer
// warps. Each takes 16 of a tile's 64 entries with a maximum, a sum and an accumulator of its own, so
// that warps meet only at an item's end: S = Q K^T and O += P V are 16 x 8 x 16 matrix instructions, P
// staying in registers between them. 16 rows of a 128-row product would be a waste that the tensor cores
// can afford, but a warp that needs no other's numbers keeps more copies in flight: 16-row products issue
// 700 of an SM's 8300 instructions a microsecond.
// Bound: the bytes of keys and values. Decode batch of 64 rows (17 to 8191 entries, 8 key heads of 128, one
// token, bf16; 1.08 GB): 172 us, 6.2 TB/s, 0.92 of the measured copy peak.
// Rounding: probabilities go to the cache's type for the product with the values (half a step of 2^-8
// or 2^-11 relative, as the output's own rounding); maxima, sums, scores and accumulators are fp32.

#include <algorithm>
#include <cmath>

#include "sv_attend.cuh"

namespace {

using sv::AttendParams;
using sv::finite2;
using sv::kFull;
using sv::value_of;

constexpr int kTileLog2 = 6, kTile = 1 << kTileLog2;   // entries of a key tile
constexpr int kWarps = 4;                      // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kConsumers = 32 * kWarps;

template <int D>
constexpr int kStageBytes = 2 * kTile * D * 2;
template <int D>
constexpr int kStageCount = D == 64 ? 6 : 3;
constexpr int kRows = 16;                      // query rows of an item
// Queries of an item, then (the queries being read) the join of the warps' accumulators: maxima and
// sums per warp and row, and two buffers of 16 rows by 16 columns per warp.
constexpr int kJoinBytes = kWarps * kRows * 8 + 2 * kWarps * kRows * 16 * 4;
template <int D>
constexpr int kScratchBytes = kRows * D * 2 > kJoinBytes ? kRows * D * 2 : kJoinBytes;
template <int D>
constexpr int kSmemBytes = 1024 + kStageCount<D> * kStageBytes<D> + kScratchBytes<D>;

template <bool F16, int D>
__global__ void __launch_bounds__(kThreads, D == 256 ? 1 : 2)
    sv_attend_kernel(const AttendParams P, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  constexpr int kStages = kStageCount<D>;
  constexpr float kBits = sv::kProbBits<F16, false>;
  extern __shared__ unsigned char dyn[];
  __shared__ __align__(8) unsigned long long full[kStages], empty[kStages];
  __shared__ int bad_stage[kStages];
  __shared__ unsigned long long masks[sv::kMaxTreeNodes];
  __shared__ long long scan[kThreads / 32];
  __shared__ sv::Plan plan;
  __shared__ int sm_flags;
  const sv::Round& R = P.R;
  const sv::Cache& C = R.C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = (sv::smem_addr(dyn) + 1023u) & ~1023u;
  const uint32_t scratch = ring + kStages * kStageBytes<D>;
  unsigned char* const scratch_p = dyn + (scratch - sv::smem_addr(dyn));
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      sv::mbar_init(sv::smem_addr(full + s), 1);
      sv::mbar_init(sv::smem_addr(empty + s), kWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  sv::make_plan<kThreads>(R, scan, &plan);

  asm volatile("griddepcontrol.launch_dependents;");   // the join kernel's CTAs, which wait for this grid's end
  if (tid == 0 && !P.by_item) P.shared[blockIdx.x].x = -1;

  sv::Walk W;
  W.begin(R, plan);
  if (warp == kWarps) {
    // ---- Producer
    sv::TileLoader T;
    T.init(C, 2, kTileLog2);
    int issued = 0;
    bool gone = false;
    while (!gone && W.next(R)) {
      const int entries = W.w.n + W.w.m;
      const int last = W.first + W.count;
      const int32_t* const table = sv::pages_of(R, W.row, W.w);
      sv::PagesAhead pages;
      pages.begin(T, C, table, W.first, last, entries, lane);
      for (int t = W.first; t < last; ++t) {
        const int p = pages.next(T, C, table, t, last, entries, lane);
        const int s = issued % kStages;
        const uint32_t bar = sv::smem_addr(full + s);
        if (issued >= kStages &&
            !__all_sync(kFull, sv::mbar_wait(sv::smem_addr(empty + s), (issued / kStages - 1) & 1))) {
          gone = true;
          break;
        }
        const unsigned go = __ballot_sync(kFull, p >= 0), out = __ballot_sync(kFull, p == -2);
        if (lane == 0) {
          bad_stage[s] = out != 0;
          sv::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(go)) << (T.rows_log2 + 7));
        }
        __syncwarp();
        if (p >= 0) T.load(C, &kmap, &vmap, t, W.head, p, lane, ring + s * kStageBytes<D>, bar);
        ++issued;
      }
    }
    sv::fill_unused(P, D, lane, 32);           // while the last tiles are computed
    // No copy is in flight when the CTA ends.
    for (int x = issued < kStages ? 0 : issued - kStages; x < issued; ++x)
      sv::mbar_wait_drain(sv::smem_addr(full + x % kStages), (x / kStages) & 1);
    return;
  }

  // ---- Consumers
  const int g = lane >> 2, t4 = lane & 3;
  const float c = P.c;
  int done = 0;                                // tiles taken from the ring
  bool lost = false;                           // a wait gave up: every result from here on is NaN
  while (W.next(R)) {
    const int n = W.w.n, m = W.w.m, entries = n + m;
    const int row0 = W.q_tile * kRows;         // query rows of the item: [row0, row0 + kRows)
    const int rows = min(kRows, m * R.group - row0);
    const char* qb = P.q + W.row * P.row_stride + static_cast<long long>(W.head) * R.group * (D * 2);
    // Queries into shared memory, zeros in the rows past the last.
    for (int x = tid; x < kRows * (D / 8); x += kConsumers) {
      const int r = x / (D / 8), ch = x % (D / 8);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) {
        const int i = (row0 + r) / R.group, hg = (row0 + r) - i * R.group;
        v = __ldg(reinterpret_cast<const uint4*>(qb + i * P.token_stride + hg * (D * 2)) + ch);
      }
      const uint32_t a = sv::swizzled(scratch + (ch >> 3) * (kRows * 128), r, ch & 7);
      *reinterpret_cast<uint4*>(scratch_p + (a - scratch)) = v;
    }
    if (tid == 0) sm_flags = 0;
    bool bad = false;
    const int last = W.first + W.count;
    const bool tail = last * kTile > n;        // the run reaches the round's own entries
    if (P.parents && tail)
      bad = !sv::tree_masks(P.parents + static_cast<size_t>(W.row) * R.N, m, masks, tid, kConsumers);
    else if (P.parents)                        // validity alone
      for (int x = tid; x < m; x += kConsumers) {
        const int p = __ldg(P.parents + static_cast<size_t>(W.row) * R.N + x);
        bad |= x == 0 ? p != -1 : (p < 0 || p >= x);
      }
    sv::named_bar_sync(1, kConsumers);
    int tok[2];                                // token of each of this thread's query rows, g and g + 8
    float mx[2], l[2], o[D / 8][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      tok[x] = min((row0 + 8 * x + g) / R.group, m - 1);
      mx[x] = -INFINITY;
      l[x] = 0.0f;
    }
#pragma unroll
    for (int y = 0; y < D / 8; ++y)
#pragma unroll
      for (int z = 0; z < 4; ++z) o[y][z] = 0.0f;
    bool odd = false;                          // values that are not finite among the round's own

    for (int t = W.first; t < last; ++t, ++done) {
      const int s = done % kStages;
      if (!lost) lost = !__all_sync(kFull, sv::mbar_wait(sv::smem_addr(full + s), (done / kStages) & 1));
      bad |= bad_stage[s] != 0;
      const int j0 = t * kTile + 16 * warp;
      if (j0 < entries && !lost) {
        const uint32_t kb = ring + s * kStageBytes<D>, vb = kb + kTile * D * 2;
        float sc[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t kf[4], qf[4];
          sv::ldsm4(kf, sv::swizzled(kb + (kk >> 2) * (kTile * 128), 16 * warp + (lane & 7) + ((lane >> 4) << 3),
                                     ((kk & 3) << 1) + ((lane >> 3) & 1)));
          sv::ldsm4(qf, sv::swizzled(scratch + (kk >> 2) * (kRows * 128), lane & 15, ((kk & 3) << 1) + (lane >> 4)));
          sv::mma<F16>(sc[0], qf, kf[0], kf[1]);
          sv::mma<F16>(sc[1], qf, kf[2], kf[3]);
        }
        const bool edge = j0 + 16 > n;         // entries of the round itself, or behind the last
        if (edge) {
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const int a = j0 + 8 * y + 2 * t4 + (z & 1) - n, i = tok[z >> 1];
              bool see = a <= i;
              if (P.parents) see = a <= 0 || (a < m && ((masks[i] >> (a - 1)) & 1));
              if (!see) sc[y][z] = -INFINITY;
            }
        }
        // Running maximum; accumulators are rescaled only when one of the warp's rows grew.
        float grow[2];
        bool any = false;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float v = fmaxf(fmaxf(sc[0][2 * x], sc[0][2 * x + 1]), fmaxf(sc[1][2 * x], sc[1][2 * x + 1]));
          v = fmaxf(v, __shfl_xor_sync(kFull, v, 1));
          v = fmaxf(v, __shfl_xor_sync(kFull, v, 2));
          grow[x] = fmaxf(mx[x], v);
          any |= grow[x] > mx[x];
        }
        if (__any_sync(kFull, any)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float f = grow[x] == mx[x] ? 1.0f : sv::ex2((mx[x] - grow[x]) * c);
            mx[x] = grow[x];
            l[x] *= f;
#pragma unroll
            for (int y = 0; y < D / 8; ++y) {
              o[y][2 * x] *= f;
              o[y][2 * x + 1] *= f;
            }
          }
        }
        uint32_t pf[4];
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float m0 = mx[x] == -INFINITY ? 0.0f : mx[x], b = F16 ? kBits : -m0 * c, sub = F16 ? m0 : 0.0f;
            const float p0 = sv::ex2(fmaf(sc[y][2 * x] - sub, c, b)), p1 = sv::ex2(fmaf(sc[y][2 * x + 1] - sub, c, b));
            l[x] += p0 + p1;
            pf[2 * y + x] = sv::pack2<F16>(p0, p1);
          }
        // Bit masks of this thread's entries that are there, and of those that are the round's own (from n on).
        auto below = [&](int j, int x) { return (j < x ? 0xffffu : 0u) | (j + 1 < x ? 0xffff0000u : 0u); };
        const int jv = j0 + 2 * t4;
        const uint32_t keep0 = edge ? below(jv, entries) : 0u, keep1 = edge ? below(jv + 8, entries) : 0u;
        const uint32_t own0 = edge ? ~below(jv, n) : 0u, own1 = edge ? ~below(jv + 8, n) : 0u;
#pragma unroll
        for (int y = 0; y < D / 16; ++y) {
          uint32_t vf[4];
          sv::ldsm4_t(vf, sv::swizzled(vb + (y >> 2) * (kTile * 128), 16 * warp + (lane & 15),
                                       ((y & 3) << 1) + (lane >> 4)));
          if (edge) {
            vf[0] = finite2<F16>(vf[0] & keep0, own0, odd);
            vf[1] = finite2<F16>(vf[1] & keep1, own1, odd);
            vf[2] = finite2<F16>(vf[2] & keep0, own0, odd);
            vf[3] = finite2<F16>(vf[3] & keep1, own1, odd);
          }
          sv::mma<F16>(o[2 * y], pf, vf[0], vf[1]);
          sv::mma<F16>(o[2 * y + 1], pf, vf[2], vf[3]);
        }
      }
      __syncwarp();
      // A warp that gave up has not seen the tile's copies land: it gives no slot back, and the producer gives up too.
      if (lane == 0 && !lost) sv::mbar_arrive(sv::smem_addr(empty + s));
    }

    // Values of the round's own entries that are not finite were left out of the products, where their
    // zero probability would have made NaN of them: they are added to the rows that attend them.
    if (__any_sync(kFull, odd)) {
      for (int j = max(n, W.first * kTile); j < min(entries, last * kTile); ++j) {
        if (((j % kTile) >> 4) != warp) continue;
        const int page = sv::cache_page(C, W.row, j);
        if (!sv::page_ok(C, page)) continue;
        const unsigned short* v = reinterpret_cast<const unsigned short*>(C.v + sv::entry_offset(C, page, W.head, j));
        const int a = j - n;
#pragma unroll
        for (int y = 0; y < D / 8; ++y)
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float f = value_of<F16>(v[8 * y + 2 * t4 + (z & 1)]);
            if (isfinite(f)) continue;
            const int i = tok[z >> 1];
            bool see = a <= i;
            if (P.parents) see = a <= 0 || ((masks[i] >> (a - 1)) & 1);
            if (see) o[y][z] += f;
          }
      }
    }
    if (bad || lost) atomicOr(&sm_flags, 1);

    // Join of the four warps: maxima and sums, then 16 columns at a time through two buffers.
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(kFull, l[x], 1);
      l[x] += __shfl_xor_sync(kFull, l[x], 2);
    }
    sv::named_bar_sync(1, kConsumers);         // the queries have been read
    float2* ml = reinterpret_cast<float2*>(scratch_p);                       // [kWarps][kRows]
    float* buf = reinterpret_cast<float*>(scratch_p + kWarps * kRows * 8);   // [2][kWarps][16][16]
    if (t4 == 0) {
      ml[warp * kRows + g] = make_float2(mx[0], l[0]);
      ml[warp * kRows + 8 + g] = make_float2(mx[1], l[1]);
    }
    sv::named_bar_sync(1, kConsumers);
    const bool nan_item = sm_flags != 0;
    float fw[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * kRows + 8 * x + g].x);
      fw[x] = mx[x] == -INFINITY ? 0.0f : sv::ex2((mx[x] - M) * c);
    }
    const bool whole = W.count == W.w.tiles;
    const int slot = 2 * blockIdx.x + (W.first == 0 ? 1 : 0);
    // This thread's place in the joined chunks: a row and two columns of each.
    const int r = tid >> 3, jc = (tid & 7) * 2;
    float jm = -INFINITY, jl = 0.0f;
    for (int w = 0; w < kWarps; ++w) jm = fmaxf(jm, ml[w * kRows + r].x);
    for (int w = 0; w < kWarps; ++w) {
      const float2 e = ml[w * kRows + r];
      jl += e.x > -INFINITY ? e.y * sv::ex2((e.x - jm) * c) : e.y;           // the latter: 0, or NaN
    }
    if (nan_item) jl = __int_as_float(0x7fffffff);
    const int i = (row0 + r) / R.group, hq = W.head * R.group + (row0 + r) - i * R.group;
    const size_t at = (static_cast<size_t>(W.row) * R.N + i) * P.Hq + hq;
    const float inv = 1.0f / jl;
#pragma unroll
    for (int y = 0; y < D / 16; ++y) {
      float* bw = buf + (y & 1) * (kWarps * 256);
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float2*>(bw + warp * 256 + (8 * e + g) * 16 + ((8 * z + 2 * t4) ^ ((g & 1) << 3))) =
              make_float2(o[2 * y + z][2 * e] * fw[e], o[2 * y + z][2 * e + 1] * fw[e]);
      sv::named_bar_sync(1, kConsumers);
      if (r >= rows) continue;
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 e = *reinterpret_cast<const float2*>(bw + w * 256 + r * 16 + (jc ^ ((r & 1) << 3)));
        s0 += e.x;
        s1 += e.y;
      }
      if (whole) {
        *reinterpret_cast<uint32_t*>(static_cast<char*>(P.out) + (at * D + 16 * y + jc) * 2) = sv::pack2<F16>(s0 * inv, s1 * inv);
      } else {
        float* part = P.part_o + (static_cast<size_t>(slot) * D + 16 * y + jc) * kRows + r;
        part[0] = s0;
        part[kRows] = s1;
      }
    }
    if ((tid & 7) == 0 && r < rows) {
      if (!whole) P.part_ml[slot * kRows + r] = make_float2(jm, jl);
      else if (P.lse) P.lse[at] = (jm * c + (log2f(jl) - kBits)) * 0.6931471805599453f;
    }
    if (tid == 0 && W.first == 0) sv::tell_shared(P, 0, W.row, W.head, W.q_tile, rows, whole, W.item_at, W.w.tiles, plan);
    sv::named_bar_sync(1, kConsumers);         // the scratch is free for the next item's queries
  }
}

// The kernel and its query tiles: 16 rows where a key head has no more, else on the wide kernel up to 128 rows,
// whole tokens. Where there are more, it can work on two tiles at once, which then read the keys and values
// once (heads of 256 have no room for two accumulators). That pays when the second reading would come from
// HBM, or when there are items for every SM that are long against their start and end; with fewer and
// shorter ones, of which many CTAs then take a part, two tiles' parts cost more than the second reading from L2.
// Lengths are on the device: the rule takes what the tables have room for, and no more than there are pages, for the
// rows' entries (24 rows of 500 to 6000 in tables for 131,072 take 56 us so, 66 by the tables alone). Two tiles are still
// taken too often where the pages have room for much more than the rows, or a batch with an item for every SM has tables
// far wider than its rows: 76 rows of 1000 entries in tables for 131,072 81 us against 67.
// Measured with 4 key heads and trees of 31 nodes, 8 query heads a key head, one tile at a time against two: 38
// rows of 2000 entries 72 against 59 us, of 32,000 619 against 475; 76 rows of 1000 76 against 84; 8 rows of
// 64,000 266 against 223, of 16,000 78 against 90, of 4000 37 against 49; 24 rows of 12,000 135 against 153, of
// 500 to 6000 61 against 74.
struct Kernel {
  bool wide;
  int tile_rows, part_rows, ways, key_log2, ctas;     // CTAs: of an SM
};
constexpr long long kBeyondL2 = 768ll << 20;           // bytes of keys and values, about six times L2
constexpr long long kLongRow = 12 << 7;                // entries of a row
Kernel kernel_for(int N, int group, const sv_paged_cache* c, long long B, int sms) {
  const int D = c->head_dim;
  if (N * group <= 16) return {false, 16, 16, 1, kTileLog2, D == 256 ? 1 : 2};
  const int rows = 128 / group * group;
  const long long pairs = B * c->heads * ((N * group + 2 * rows - 1) / (2 * rows));
  const long long pages = B * c->max_pages < c->num_pages ? B * c->max_pages : c->num_pages;
  const long long entries = std::min<long long>(c->max_pages, c->num_pages) * c->page_size;
  const long long bytes = pages * c->page_size * c->heads * D * 4;
  const bool two = N * group > rows && D < 256 && ((pairs >= sms && entries >= kLongRow) || bytes >= kBeyondL2);
  return {true, rows, 128, two ? 2 : 1, D == 256 ? 6 : 7, 1};
}
constexpr int kMaxSms = 160;
constexpr size_t kSharedBytes = 2 * kMaxSms * sizeof(int4);   // two ways or two CTAs an SM

template <bool F16, int D>
int launch(const AttendParams& P, const CUtensorMap& k, const CUtensorMap& v, int grid, cudaStream_t st) {
  auto kern = sv_attend_kernel<F16, D>;
  static std::atomic<unsigned long long> allowed{0};
  if (sv::allow_shared(kern, kSmemBytes<D>, allowed) != SV_OK) return SV_ERR_CUDA;
  kern<<<grid, kThreads, kSmemBytes<D>, st>>>(P, k, v);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace

extern "C" size_t spec_verify_paged_attention_workspace_size(int32_t N, int32_t Hq,
                                                             const sv_paged_cache* cache) {
  if (!cache || N < 1 || N > SV_MAX_GAMMA + 1 || Hq < 1 || Hq > 1024 || cache->heads < 1 ||
      Hq % cache->heads != 0 || Hq / cache->heads > 128 || cache->head_dim < 1 || cache->head_dim > 256)
    return 0;
  // Two query tiles' parts where two could be worked on at once, whatever the batch.
  const Kernel k = kernel_for(N, Hq / cache->heads, cache, 1 << 20, 1);
  const size_t part = static_cast<size_t>(k.ways) * k.part_rows * (cache->head_dim * 4 + 8);
  return kSharedBytes + (2 * k.ctas * kMaxSms * part + 255) / 256 * 256;
}

extern "C" int spec_verify_paged_attention(const void* q, int64_t q_row_stride,
                                           int64_t q_token_stride, const sv_paged_cache* cache,
                                           const int32_t* prefix_len, const int32_t* num_queries,
                                           const int32_t* tree_parents, float scale, void* out,
                                           float* out_lse, int32_t B, int32_t N, int32_t Hq,
                                           void* workspace, size_t workspace_bytes,
                                           void* cuda_stream) {
  AttendParams P;
  int st = sv::check_cache(cache, B, false, &P.R.C);
  if (st != SV_OK) return st;
  if (!q || !prefix_len || !out) return SV_ERR_NULL_POINTER;
  st = sv::check_tokens(q, q_row_stride, q_token_stride, B, N, Hq, cache->head_dim);
  if (st != SV_OK) return st;
  if (Hq % cache->heads != 0 || Hq / cache->heads > 128 || !(scale > 0.0f) || !std::isfinite(scale)) return SV_ERR_BAD_SHAPE;
  if (sv::misaligned(out, 16) || sv::misaligned(out_lse, 4) || sv::misaligned(prefix_len, 4) ||
      sv::misaligned(num_queries, 4) || sv::misaligned(tree_parents, 4) ||
      sv::misaligned(workspace, 256))
    return SV_ERR_MISALIGNED;
  const size_t need = spec_verify_paged_attention_workspace_size(N, Hq, cache);
  if (!workspace || workspace_bytes < need) return SV_ERR_WORKSPACE_TOO_SMALL;
  const unsigned long long rows = 4ull * B, tokens = rows * N * Hq;
  if (sv::overlap({{out, tokens / 2 * cache->head_dim}, {out_lse, tokens}, {workspace, need}},
                  {sv::tokens_of(q, q_row_stride, q_token_stride, B, N, Hq, cache->head_dim), {prefix_len, rows},
                   {num_queries, rows}, {tree_parents, rows * N}, sv::table_of(cache, B),
                   sv::weights_of(cache), sv::pages_of(cache, cache->k), sv::pages_of(cache, cache->v)}))
    return SV_ERR_OVERLAP;
  int dev = 0;
  st = sv::current_device_status(&dev);
  if (st != SV_OK) return st;
  const int D = cache->head_dim, group = Hq / cache->heads;
  int sms = sv::device_sms(dev);
  if (sms < 1) return SV_ERR_CUDA;
  if (sms > kMaxSms) sms = kMaxSms;
  const Kernel k = kernel_for(N, group, cache, B, sms);
  CUtensorMap kmap, vmap;
  st = sv::cache_tensor_map(cache, cache->k, sv::box_rows(cache), &kmap);
  if (st == SV_OK) st = sv::cache_tensor_map(cache, cache->v, sv::box_rows(cache), &vmap);
  if (st != SV_OK) return st;
  P.R.prefix = prefix_len;
  P.R.num = num_queries;
  P.R.B = B;
  P.R.N = N;
  P.R.group = group;
  P.R.q_rows = k.tile_rows * k.ways;
  P.R.tile_log2 = k.key_log2;
  P.R.extra = k.wide ? 2 : 1;
  P.R.none_ok = false;
  P.q = static_cast<const char*>(q);
  P.row_stride = q_row_stride * 2;
  P.token_stride = q_token_stride * 2;
  P.parents = tree_parents;
  P.out = out;
  P.lse = out_lse;
  P.c = scale * sv::kLog2e;
  P.Hq = Hq;
  P.tile_rows = k.tile_rows;
  P.ways = k.ways;
  // As many CTAs as the GPU holds, or as many as the batch can have tiles.
  const long long tile = 1 << P.R.tile_log2;
  const long long items = static_cast<long long>(B) * cache->heads * ((N * group + P.R.q_rows - 1) / P.R.q_rows);
  const long long most = items * ((static_cast<long long>(cache->max_pages) * cache->page_size + tile - 1) / tile);
  const int grid = static_cast<int>(most < sms * k.ctas ? most : sms * k.ctas);
  // Few items against the CTAs: each has many parts, and their records are by item.
  const int tiles = (N * group + k.tile_rows - 1) / k.tile_rows;
  P.by_item = static_cast<long long>(B) * cache->heads * tiles * 4 <= grid ? tiles : 0;
  char* ws = static_cast<char*>(workspace);
  P.shared = reinterpret_cast<int4*>(ws);
  ws += kSharedBytes;
  P.part_ml = reinterpret_cast<float2*>(ws);
  P.part_o = reinterpret_cast<float*>(ws + static_cast<size_t>(2) * grid * k.ways * k.part_rows * 8);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool f16 = cache->dtype == SV_DTYPE_F16;
  if (k.wide) {
    CUtensorMap qmap;
    const int tokens = k.tile_rows / group < N ? k.tile_rows / group : N;
    st = sv::query_tensor_map(q, q_row_stride, q_token_stride, B, N, Hq, D, cache->dtype, group, tokens, &qmap);
    if (st != SV_OK) return st;
    st = sv::launch_attend_wide(P, f16, kmap, vmap, qmap, tokens, grid, s);
  }
  else if (D == 64) st = f16 ? launch<true, 64>(P, kmap, vmap, grid, s) : launch<false, 64>(P, kmap, vmap, grid, s);
  else if (D == 128) st = f16 ? launch<true, 128>(P, kmap, vmap, grid, s) : launch<false, 128>(P, kmap, vmap, grid, s);
  else st = f16 ? launch<true, 256>(P, kmap, vmap, grid, s) : launch<false, 256>(P, kmap, vmap, grid, s);
  return st == SV_OK ? sv::launch_attend_join(P, f16, k.wide, grid, s) : st;
}
