// Attention of a round's tokens in a batch whose rows share the fronts of their contexts (a common prompt or document;
// [R] "Speculative decoding", rayaq.ca ml-models -- Verification attention and the cache).
//
// A row's entries are those that its group shares, A, and its own, B. With m = max s_ij, l = sum exp(s_ij - m) and
// o = sum exp(s_ij - m) v_j over each of the two,
//   M = max(m_A, m_B),  L = l_A e^(m_A - M) + l_B e^(m_B - M),  out = (o_A e^(m_A - M) + o_B e^(m_B - M)) / L.
// A of all the group's rows and tokens is one set of products with the group's keys and values, read once for up to
// 128 or 256 query rows, not once a row. One launch of the wide kernel (sv_attend_wide.cuh) does the fronts and the
// rows' own entries, cut into runs of equal time, whose results, of several CTAs where an item is cut, the merge kernel
// here puts together, a query or four a warp.
// Bound: the bytes of the entries, each read once, or for large groups the products (4 D a query head and entry). 64 rows
// of one token over 8000 shared and 17 to 1000 own entries, 32/8 heads of 128: 54 us (floor 25; 225 by rows that each read
// all of it): 41 to 46 of the attention, of which about 14 are its start and end, then the merge.
// Two launches of each (the fronts, their join, the rows' own entries with the front added at an item's end, their join)
// took 99 us: each launch's start and end cost more than the rows' own entries gained by kernels of their own.
// Rounding: the sides are fp32 sums and maxima; the output is rounded once.

#include <algorithm>

#include "sv_attend_wide.cuh"

namespace {

using sv::SharedParams;

// The tokens that are used, row after row, so that a front's query tiles have no others: 64 rows of 9 tokens, of which 62%
// are used, over two prompts 85 us so, 92 without. CTA (b, y) copies every gridDim.y-th token of row b.
constexpr int kPackThreads = 256, kMaxPacked = 1024;   // (each CTA sums up the rows before its own)
__global__ void __launch_bounds__(kPackThreads) sv_attend_pack_kernel(const SharedParams P, int32_t* first, uint4* packed, int words) {
  asm volatile("griddepcontrol.launch_dependents;");
  const sv::SharedRound& R = P.R;
  const int b = blockIdx.x, tid = threadIdx.x;
  int n, m, sum = 0;
  auto tokens = [&](int row) { return sv::round_lengths(R.C, R.prefix, R.num, row, R.N, false, &n, &m) ? m : 0; };
  const int mine = tokens(b);
  for (int r = tid; r < b; r += kPackThreads) sum += tokens(r);
  __shared__ int warps[kPackThreads / 32];
  sum = __reduce_add_sync(kFull, sum);
  if ((tid & 31) == 0) warps[tid >> 5] = sum;
  __syncthreads();
  int at = 0;
#pragma unroll
  for (int w = 0; w < kPackThreads / 32; ++w) at += warps[w];
  if (blockIdx.y == 0 && tid == 0) {
    first[b] = at;
    if (b + 1 == R.B) first[R.B] = at + mine;
  }
  for (int i = blockIdx.y; i < mine; i += gridDim.y) {
    const uint4* from = reinterpret_cast<const uint4*>(P.q + b * P.row_stride + i * P.token_stride);
    uint4* to = packed + static_cast<size_t>(at + i) * words;
#pragma unroll 4
    for (int x = tid; x < words; x += kPackThreads) to[x] = __ldg(from + x);
  }
}

template <int kQueries>
constexpr int kMergeWarps = kQueries == 1 ? 16 : 8;
// What the plan takes a tile and an item (its queries and its end) to cost, in units of 0.25 us: a tile on two ways 2 us,
// on one about what its bytes take from HBM among other CTAs' products. (All tiles alike and an item two of them: 64 rows
// of one token over 8000 shared entries 78 us against 61, two prompts' rounds of 9 tokens 113 against 92. One-way tiles at
// 3 or 5 units, items at 6 to 20: 61 to 65 and 93 to 98.)
constexpr int kTwoWays = 8, kOneWay = 4, kOneItem = 10, kTwoItem = 15;

// A warp has kQueries of a key head's query heads at one token: they have the same items, and rows of these that follow
// one another. Or `across` warps have one query: they divide its parts and sides among them and meet in shared memory.
template <bool F16, int D, int kQueries>
__global__ void __launch_bounds__(32 * kMergeWarps<kQueries>) sv_attend_merge_kernel(const SharedParams P, int across) {
  constexpr int kCols = D / 32;
  constexpr int kWarps = kMergeWarps<kQueries>;
  __shared__ float acc[kQueries == 1 ? kWarps : 1][D];
  __shared__ float2 ml[kWarps];
  const sv::SharedRound& R = P.R;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = kQueries == 1 ? warp % across : 0;
  const int bunches = (R.group + kQueries - 1) / kQueries, all_bunches = R.B * R.N * R.C.heads * bunches;
  const int id = kQueries == 1 ? blockIdx.x * (kWarps / across) + warp / across : blockIdx.x * kWarps + warp;
  const bool there = id < all_bunches;
  const int x = there ? id : 0, th = x / bunches, h0 = (x - th * bunches) * kQueries;   // its first query head of the key head's
  const int token = th / R.C.heads, head = th - token * R.C.heads, b = token / R.N, i = token - b * R.N;
  const int queries = min(kQueries, R.group - h0);
  const size_t out_at = static_cast<size_t>(token) * P.Hq + head * R.group + h0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 row = __ldcg(P.rows + b);
  const int own = R.first_token(b) + i;        // its place among the tokens of q
  const size_t at = static_cast<size_t>(own) * P.Hq + head * R.group + h0;
  const int m = __ldcg(P.bad_groups) == 0 ? row.x : -1, s = row.w;
  float v[kQueries][kCols], M[kQueries], L[kQueries];
#pragma unroll
  for (int q = 0; q < kQueries; ++q) {
    M[q] = -INFINITY;
    L[q] = 0.0f;
#pragma unroll
    for (int y = 0; y < kCols; ++y) v[q][y] = 0.0f;
  }
  if (there && i < m) {
    // Where the two items have their records, and the first query's row of their query tiles.
    int row_front = 0, tile_front = 0;
    const int row_own = i * R.group + h0;
    const int2 oo = __ldcg(P.records + P.record_at(R.groups + b, head, 0, 0));
    int2 of = make_int2(0, -1);
    if (s > 0) {
      row_front = (own - row.z) * R.group + h0;
      tile_front = row_front / P.tile_rows;
      row_front -= tile_front * P.tile_rows;
      of = __ldcg(P.records + P.record_at(row.y, head, tile_front, row.z));
    }
    const int fronts = of.x < 0 ? 1 : of.y - of.x + 1, all = fronts + (oo.x < 0 ? 1 : oo.y - oo.x + 1);
    // The k-th result's first row: a side's, or part k's of those that share the item (the first of them is the later
    // of its CTA's two).
    const int part = P.ways * 128;
    const size_t row_a = of.x < 0 ? P.side_at(0, at) : static_cast<size_t>(2 * of.x * part + tile_front % P.ways * 128 + row_front);
    const size_t row_b = oo.x < 0 ? P.side_at(1, at) : static_cast<size_t>(2 * oo.x * part + row_own);
    const float* const o_a = (of.x < 0 ? P.side_o : P.part_o) + row_a * D;
    const float* const o_b = (oo.x < 0 ? P.side_o : P.part_o) + row_b * D;
    const float2* const ml_a = (of.x < 0 ? P.side_ml : P.part_ml) + row_a;
    const float2* const ml_b = (oo.x < 0 ? P.side_ml : P.part_ml) + row_b;
    constexpr int kBatch = kQueries == 1 ? 4 : 1;        // results in flight together
    for (int k0 = mine; k0 < all; k0 += kBatch * across) {
      float2 e[kBatch][kQueries], z[kBatch][kQueries][kCols / 2];
#pragma unroll
      for (int y = 0; y < kBatch; ++y) {
        const int k = k0 + y * across;
        if (k >= all) break;
        const bool front = k < fronts;
        const int j = front ? k : k - fronts, off = (front ? of.x : oo.x) < 0 ? 0 : (2 * j + (j == 0)) * part;
        const float2* const o = reinterpret_cast<const float2*>((front ? o_a : o_b) + off * D) + lane;
        const float2* const ml = (front ? ml_a : ml_b) + off;
#pragma unroll
        for (int q = 0; q < kQueries; ++q) {
          if (q >= queries) break;
          e[y][q] = __ldcg(ml + q);
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) z[y][q][c] = __ldcg(o + q * (D / 2) + 32 * c);
        }
      }
#pragma unroll
      for (int y = 0; y < kBatch; ++y) {
        if (k0 + y * across >= all) break;
#pragma unroll
        for (int q = 0; q < kQueries; ++q) {
          if (q >= queries) break;
          const float2 g = e[y][q];
          const float top = fmaxf(M[q], g.x);
          const float f = M[q] == top ? 1.0f : (M[q] == -INFINITY ? 0.0f : sv::ex2((M[q] - top) * P.c));
          const float t = g.x == -INFINITY ? 0.0f : sv::ex2((g.x - top) * P.c);
          M[q] = top;
          L[q] = L[q] * f + (g.x == -INFINITY ? g.y : g.y * t);          // the former: 0, or NaN
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) {  // (an infinity times a weight of 0: NaN)
            v[q][2 * c] = v[q][2 * c] * f + z[y][q][c].x * t;
            v[q][2 * c + 1] = v[q][2 * c + 1] * f + z[y][q][c].y * t;
          }
        }
      }
    }
  }
  if (kQueries == 1 && across > 1) {
#pragma unroll
    for (int y = 0; y < kCols / 2; ++y) *reinterpret_cast<float2*>(&acc[warp][2 * lane + 64 * y]) = make_float2(v[0][2 * y], v[0][2 * y + 1]);
    if (lane == 0) ml[warp] = make_float2(M[0], L[0]);
    __syncthreads();
    if (mine > 0) return;
    for (int k = 1; k < across; ++k) M[0] = fmaxf(M[0], ml[warp + k].x);
    L[0] = 0.0f;
#pragma unroll
    for (int y = 0; y < kCols; ++y) v[0][y] = 0.0f;
    for (int k = 0; k < across; ++k) {
      const float2 e = ml[warp + k];
      const float t = e.x == -INFINITY ? 0.0f : sv::ex2((e.x - M[0]) * P.c);
      L[0] += e.x == -INFINITY ? e.y : e.y * t;
#pragma unroll
      for (int y = 0; y < kCols / 2; ++y) {
        const float2 z = *reinterpret_cast<const float2*>(&acc[warp + k][2 * lane + 64 * y]);
        v[0][2 * y] += z.x * t;
        v[0][2 * y + 1] += z.y * t;
      }
    }
  }
  if (!there) return;
  const bool some = i < m;
  const float none = m >= 0 ? 0.0f : __int_as_float(0x7fffffff);
#pragma unroll
  for (int q = 0; q < kQueries; ++q) {
    if (q >= queries) break;
    const float inv = 1.0f / L[q];
    uint32_t* out = reinterpret_cast<uint32_t*>(P.out) + (out_at + q) * (D / 2) + lane;
#pragma unroll
    for (int y = 0; y < kCols / 2; ++y)
      out[32 * y] = some ? sv::pack2<F16>(v[q][2 * y] * inv, v[q][2 * y + 1] * inv) : sv::pack2<F16>(none, none);
    if (P.lse && lane == 0)
      P.lse[out_at + q] = some ? (M[q] * P.c + (log2f(L[q]) - sv::kProbBits<F16, true>)) * 0.6931471805599453f : none;
  }
}

template <bool F16, int D, int kQueries>
int merge(const SharedParams& P, int across, cudaStream_t st) {
  const long long warps = static_cast<long long>(P.R.B) * P.R.N * P.R.C.heads * ((P.R.group + kQueries - 1) / kQueries) * across;
  return sv::launch_ahead(sv_attend_merge_kernel<F16, D, kQueries>, dim3(static_cast<unsigned>((warps - 1) / kMergeWarps<kQueries> + 1)),
                          32 * kMergeWarps<kQueries>, 0, st, P, across);
}
template <bool F16, int D>
int merge(const SharedParams& P, int sms, cudaStream_t st) {
  // Up to as many warps as the GPU holds at once (32 an SM): few queries, whose fronts may be in many parts, have up to
  // sixteen each.
  const long long queries = static_cast<long long>(P.R.B) * P.R.N * P.Hq, most = 32ll * sms;
  if (queries > most) return merge<F16, D, 4>(P, 1, st);
  int across = 16;
  while (across > 1 && queries * across > most) across /= 2;
  return merge<F16, D, 1>(P, across, st);
}
template <bool F16>
int merge(const SharedParams& P, int sms, cudaStream_t st) {
  const int D = P.R.C.head_dim;
  return D == 64 ? merge<F16, 64>(P, sms, st) : (D == 128 ? merge<F16, 128>(P, sms, st) : merge<F16, 256>(P, sms, st));
}

constexpr int kMaxSms = 160;
// Query heads times room from which a third launch is worth the products that it saves (a third of 2 us for 256 query rows
// and 128 entries, over the SMs: about 5 us).
constexpr long long kWorthPacking = 1ll << 25;
constexpr size_t kFlagBytes = 256;
size_t rounded(size_t bytes) { return (bytes + 255) / 256 * 256; }
// Tokens packed, and the rows' first ones.
bool packs(int B, int N) { return N > 1 && B <= kMaxPacked; }
size_t packed_bytes(int B, int N, int Hq, int D) {
  return packs(B, N) ? rounded(static_cast<size_t>(B + 1) * 4) + rounded(static_cast<size_t>(B) * N * Hq * D * 2) : 0;
}
// Entries of a row; bytes of all rows' keys and values.
constexpr long long kShortRoom = 512, kLittleRoom = 48ll << 20, kSomeRoom = 256ll << 20, kMuchRoom = 640ll << 20;
constexpr long long kMaxQueries = 1ll << 28;   // query heads of all tokens

bool sizes_ok(int32_t B, int32_t N, int32_t Hq, const sv_paged_cache* c) {
  return B >= 1 && B <= (1 << 20) && N >= 1 && N <= SV_MAX_GAMMA + 1 && Hq >= 1 && Hq <= 1024 && c->heads >= 1 &&
         Hq % c->heads == 0 && Hq / c->heads <= 128 && static_cast<long long>(B) * N * Hq <= kMaxQueries;
}
int rows_of_tile(int group) { return 128 / group * group; }   // query rows of a query tile: whole tokens
size_t part_rows(int D) { return static_cast<size_t>(2 * kMaxSms) * (D < 256 ? 2 : 1) * 128; }
// Query tiles of a key head's fronts, at most (each group's last may be short).
long long front_tiles(long long queries, int groups, int group) { return queries / rows_of_tile(group) + groups + 1; }

}  // namespace

namespace sv {

int launch_attend_shared(const SharedParams& P, bool f16, const CUtensorMap& k, const CUtensorMap& v,
                         const CUtensorMap& q, int q_tokens, int grid, cudaStream_t st) {
  return f16 ? launch_type<true, true>(P, k, v, q, q_tokens, grid, st) : launch_type<false, true>(P, k, v, q, q_tokens, grid, st);
}

}  // namespace sv

extern "C" size_t spec_verify_shared_attention_workspace_size(int32_t B, int32_t N, int32_t Hq, int32_t groups,
                                                              const sv_paged_cache* cache) {
  if (!cache || !sizes_ok(B, N, Hq, cache) || cache->head_dim < 1 || cache->head_dim > 256 || groups < 1 || groups > (1 << 20)) return 0;
  const int D = cache->head_dim, heads = cache->heads, group = Hq / heads;
  if (N * group > rows_of_tile(group)) return spec_verify_paged_attention_workspace_size(N, Hq, cache);   // rows go by themselves
  const size_t row = D * 4 + 8, queries = static_cast<size_t>(B) * N * Hq;
  const size_t records = static_cast<size_t>(heads) * (B + front_tiles(static_cast<long long>(B) * N * group, groups, group));
  return std::max(spec_verify_paged_attention_workspace_size(N, Hq, cache),
                  kFlagBytes + rounded(static_cast<size_t>(B) * sizeof(int4)) + rounded(records * sizeof(int2)) +
                      rounded(part_rows(D) * row) + rounded(2 * queries * row) + packed_bytes(B, N, Hq, D));
}

extern "C" int spec_verify_shared_attention(const void* q, int64_t q_row_stride, int64_t q_token_stride,
                                            const sv_paged_cache* cache, const int32_t* prefix_len,
                                            const int32_t* shared_len, const int32_t* group_start, int32_t groups,
                                            const int32_t* num_queries, const int32_t* tree_parents, float scale, void* out,
                                            float* out_lse, int32_t B, int32_t N, int32_t Hq, void* workspace,
                                            size_t workspace_bytes, void* cuda_stream) {
  sv::Cache C;
  int st = sv::check_cache(cache, B, false, &C);
  if (st != SV_OK) return st;
  if (!q || !prefix_len || !shared_len || !group_start || !out) return SV_ERR_NULL_POINTER;
  st = sv::check_tokens(q, q_row_stride, q_token_stride, B, N, Hq, cache->head_dim);
  if (st != SV_OK) return st;
  if (!sizes_ok(B, N, Hq, cache) || groups < 1 || groups > (1 << 20) || !(scale > 0.0f) || !std::isfinite(scale)) return SV_ERR_BAD_SHAPE;
  if (B > 1 && N > 1 && q_row_stride != N * q_token_stride) return SV_ERR_BAD_SHAPE;
  if (sv::misaligned(out, 16) || sv::misaligned(out_lse, 4) || sv::misaligned(prefix_len, 4) ||
      sv::misaligned(shared_len, 4) || sv::misaligned(group_start, 4) || sv::misaligned(num_queries, 4) ||
      sv::misaligned(tree_parents, 4) || sv::misaligned(workspace, 256))
    return SV_ERR_MISALIGNED;
  const size_t need = spec_verify_shared_attention_workspace_size(B, N, Hq, groups, cache);
  if (!workspace || workspace_bytes < need) return SV_ERR_WORKSPACE_TOO_SMALL;
  const unsigned long long rows = 4ull * B, tokens = rows * N * Hq;
  if (sv::overlap({{out, tokens / 2 * cache->head_dim}, {out_lse, tokens}, {workspace, need}},
                  {sv::tokens_of(q, q_row_stride, q_token_stride, B, N, Hq, cache->head_dim), {prefix_len, rows},
                   {shared_len, rows}, {group_start, 4ull * groups + 4}, {num_queries, rows}, {tree_parents, rows * N},
                   sv::table_of(cache, B), sv::weights_of(cache), sv::pages_of(cache, cache->k), sv::pages_of(cache, cache->v)}))
    return SV_ERR_OVERLAP;
  int dev = 0;
  st = sv::current_device_status(&dev);
  if (st != SV_OK) return st;
  int sms = sv::device_sms(dev);
  if (sms < 1) return SV_ERR_CUDA;
  if (sms > kMaxSms) sms = kMaxSms;
  const int D = cache->head_dim, group = Hq / cache->heads, rows_tile = rows_of_tile(group);
  // A group's queries fill the query tiles that its front is read for. Where a row's queries alone fill much of one, fronts
  // gain less, the second reading of their entries coming from L2 or hiding behind the products; and the kernel's start and
  // end and the merge take longer. So rows go by themselves where they have more than a query tile, and else by the room
  // that the tables and pages have for their entries (lengths are on the device). Fronts against rows, us, up to 600 entries
  // a row's own: 32/8 heads of 128, one token a row: 4 rows over 512 shared entries 17 and 13, over 8192 20 and 26; 64 rows
  // over 256 33 and 27, over 1024 34 and 44. 4 key heads of 128: 36 query rows, 24 rows over 4000 40 and 43, over 32,000 77
  // and 188; 72 query rows 52 and 43, 122 and 190, 64 rows over 4000 69 and 82; 128 query rows, 64 rows over 4000 95 and 86,
  // over 32,000 390 and 474. 16/2 heads of 64, one token: 64 rows over 1024 21 and 17, over 4096 23 and 30. One key head of
  // 256, one token: 4 rows over 512 15 and 15, over 2048 16 and 17. The room is the tables', so that short rows in tables of
  // a long context go by fronts: 4 rows over 512 in tables of 32,768 20 and 16, 24 rows of 18 tokens over 1000, 16/4 heads, 38
  // and 27, 64 of 32 over 1000, 8/2 heads, 46 and 33. (More than a query tile a row: not measured by fronts, a row's own
  // entries have one record and one query tile.)
  const long long room = std::min<long long>(cache->max_pages, cache->num_pages) * cache->page_size;
  const long long little = N * group > 96 ? kMuchRoom : (N * group > 64 ? kSomeRoom : (D < 256 ? kLittleRoom : kLittleRoom / 4));
  if (N * group > rows_tile || (D < 256 && room <= kShortRoom) || B * room * cache->heads * D * 4 <= little)
    return spec_verify_paged_attention(q, q_row_stride, q_token_stride, cache, prefix_len, num_queries, tree_parents, scale, out,
                                       out_lse, B, N, Hq, workspace, workspace_bytes, cuda_stream);
  // Two query tiles at once where groups, the empty ones among them, have more than one's rows on average (they are on the
  // device). Two at once and one, us: a group of 256 rows of one token over 32,000 186 and 207, 1024 rows over 8000 363 and
  // 373, 64 of 9 over 16,000 142 and 140, 40 of 5 over 4000 49 and 45, 256 of 2 over 16,000, 64/8 heads of 64, 249 and 236;
  // groups below a tile: 40 of 3 rows over 4000 127 and 117, 16 of 4 rows of 4 tokens over 3000 68 and 64.
  const long long all = static_cast<long long>(B) * N * group;
  const int ways = D < 256 && all > static_cast<long long>(groups) * rows_tile ? 2 : 1;
  const int q_tokens = static_cast<int>(std::min<long long>(rows_tile / group, static_cast<long long>(B) * N));
  CUtensorMap kmap, vmap, qmap;
  st = sv::cache_tensor_map(cache, cache->k, sv::box_rows(cache), &kmap);
  if (st == SV_OK) st = sv::cache_tensor_map(cache, cache->v, sv::box_rows(cache), &vmap);
  if (st != SV_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  SharedParams P;
  P.R.C = C;
  P.R.prefix = prefix_len;
  P.R.num = num_queries;
  P.R.B = B;
  P.R.N = N;
  P.R.group = group;
  P.R.none_ok = false;
  P.R.start = group_start;
  P.R.common = shared_len;
  P.R.groups = groups;
  P.out = out;
  P.lse = out_lse;
  P.Hq = Hq;
  P.R.q_rows = rows_tile * ways;
  P.R.tile_log2 = D == 256 ? 6 : 7;
  P.R.one_rows = ways == 2 ? rows_tile : static_cast<int>(kMaxQueries);
  P.R.one_units = kOneWay;
  P.R.two_units = ways == 2 ? kTwoWays : kOneWay;
  P.R.extra = kOneItem;
  P.R.two_extra = kTwoItem;
  P.q = static_cast<const char*>(q);
  P.row_stride = q_row_stride * 2;
  P.token_stride = q_token_stride * 2;
  P.parents = tree_parents;
  P.c = scale * sv::kLog2e;
  P.tile_rows = rows_tile;
  P.ways = ways;
  P.by_item = 0;
  P.front_tiles = static_cast<int>(front_tiles(all, groups, group));
  // As many CTAs as the GPU holds, or as many as the batch can have tiles.
  const long long tile = 1 << P.R.tile_log2;
  const long long items = static_cast<long long>(cache->heads) * (B + P.front_tiles);
  const long long most = items * ((static_cast<long long>(cache->max_pages) * cache->page_size + tile - 1) / tile);
  const int grid = static_cast<int>(std::min<long long>(most, sms));
  char* ws = static_cast<char*>(workspace);
  P.shared = nullptr;
  P.bad_groups = reinterpret_cast<int*>(ws);
  ws += kFlagBytes;
  P.rows = reinterpret_cast<int4*>(ws);
  ws += rounded(static_cast<size_t>(B) * sizeof(int4));
  P.records = reinterpret_cast<int2*>(ws);
  ws += rounded(static_cast<size_t>(items) * sizeof(int2));
  P.part_o = reinterpret_cast<float*>(ws);
  P.part_ml = reinterpret_cast<float2*>(P.part_o + part_rows(D) * D);
  ws += rounded(part_rows(D) * (D * 4 + 8));
  P.side_o = reinterpret_cast<float*>(ws);
  P.side_ml = reinterpret_cast<float2*>(P.side_o + static_cast<size_t>(2) * B * N * Hq * D);
  ws += rounded(static_cast<size_t>(2) * B * N * Hq * (D * 4 + 8));
  const bool f16 = cache->dtype == SV_DTYPE_F16, packed = num_queries && packs(B, N) && all * cache->heads * room >= kWorthPacking;
  int32_t* const first = reinterpret_cast<int32_t*>(ws);
  uint4* const tokens_to = reinterpret_cast<uint4*>(ws + rounded(static_cast<size_t>(B + 1) * 4));
  P.R.first = packed ? first : nullptr;
  st = packed ? sv::query_tensor_map(tokens_to, 0, static_cast<int64_t>(Hq) * D, 1, B * N, Hq, D, cache->dtype, group, q_tokens, &qmap)
              : sv::query_tensor_map(q, 0, N > 1 ? q_token_stride : q_row_stride, 1, B * N, Hq, D, cache->dtype, group, q_tokens, &qmap);
  if (st != SV_OK) return st;
  if (packed) {
    sv_attend_pack_kernel<<<dim3(B, std::min(N, 4)), kPackThreads, 0, s>>>(P, first, tokens_to, Hq * D / 8);
    if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  }
  st = sv::launch_attend_shared(P, f16, kmap, vmap, qmap, q_tokens, grid, s);
  if (st != SV_OK) return st;
  return f16 ? merge<true>(P, sms, s) : merge<false>(P, sms, s);
}
