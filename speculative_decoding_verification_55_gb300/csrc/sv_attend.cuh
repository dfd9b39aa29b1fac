// What the two attention kernels share: their arguments and the handling of values that are not finite.
#pragma once

#include "sv_tiles.cuh"

namespace sv {

template <bool kShared>
struct AttendParamsOf {
  typename Batch<kShared>::Rows R;
  const char* q;
  long long row_stride, token_stride;          // bytes
  const int32_t* parents;
  void* out;
  float* lse;
  float c;                                     // scale * log2(e)
  int Hq;
  int tile_rows, ways;                         // query rows of a query tile, query tiles of an item
  // Items that several CTAs share leave a part each, which the join kernel puts together. An item's
  // first part is part 2 p + 1 of the CTA p that holds its first tile, the others part 2 p of theirs, each a
  // tile of rows per way.
  int by_item;                                 // query tiles of a row and head, where records are by item
  int4* shared;                                // [grid][ways] the shared item whose first tile a CTA holds: row
                                               // (-1: none), head, 256 x query tile + its rows, the last CTA; or
                                               // by item: the first CTA (-1: it is whole), 0, rows, the last CTA
  float* part_o;                               // [2 grid][ways][D][rows]
  float2* part_ml;                             // [2 grid][ways][rows] maximum and sum
};
typedef AttendParamsOf<false> AttendParams;

// Of rows that share fronts. An item's result, of a query tile of 128 rows, is sums, a maximum and a sum of weights a
// row: where a CTA has all of it, at its queries' place on a side (0: the fronts', 1: the rows' own entries'), else in a
// part each of the CTAs that share it. Every item leaves a record; the merge kernel puts the parts and sides of each
// query together.
struct SharedParams : AttendParamsOf<true> {
  float* side_o;                               // [2][B N Hq][D]
  float2* side_ml;                             // [2][B N Hq] maximum and sum
  int2* records;                               // (by record_at) first and last CTA; first -1: one CTA has all of it
  int4* rows;                                  // [B] a row's tokens (-1: in error), its group, the group's first token, shared_len
  int* bad_groups;                             // not 0: group_start does not ascend within 0 .. B
  int front_tiles;                             // records of a key head's fronts (a row's key head has one: one query tile)
  __device__ __forceinline__ size_t side_at(int side, size_t at) const {
    return static_cast<size_t>(side) * R.B * R.N * Hq + at;
  }
  // The rows' records, then the fronts': group g, whose first token is token0, has its from token0 x group / tile_rows
  // + g on (its last query tile may be short, which the + g makes up for).
  __device__ __forceinline__ size_t record_at(int row, int head, int q_tile, int token0) const {
    if (row >= R.groups) return static_cast<size_t>(row - R.groups) * R.C.heads + head;
    return static_cast<size_t>(R.B) * R.C.heads + static_cast<size_t>(head) * front_tiles +
           token0 * R.group / tile_rows + row + q_tile;
  }
};
template <bool kShared>
using ParamsOf = typename std::conditional<kShared, SharedParams, AttendParams>::type;

// Probabilities are kept times a power of two: relative to a row's running maximum they go down to 2^-25 and less in
// long rows, and a half's steps below 2^-14 are all 2^-24. The largest are 2^15 (a half ends at 65,504): the 16-row
// kernel's maximum is the true one, the wide kernel's may lag by kSlack, which leaves it 2^7, half a step of 2^-32 of the
// maximum. (A slack of 2^4 and a factor of 2^11 cost a long row 1.2 of 39 us.) Accumulators and sums have the factor too;
// it leaves with their quotient and is taken out of the lse. So near a half's end, the maximum is subtracted from a score
// before the product with c, which is exact for the largest: c s - c m of scores in the tens of millions is off by more
// than 1. (That costs two query tiles at once 520 against 504 us for 38 rows of 32,000 entries, and no other case measured.)
// bf16 has fp32's exponents and needs neither.
constexpr float kSlack = 8.0f;
template <bool F16, bool kWide>
constexpr float kProbBits = F16 ? (kWide ? 15.0f - kSlack : 15.0f) : 0.0f;

template <bool F16>
__device__ __forceinline__ float value_of(uint32_t h) {
  if (F16) return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
  return __uint_as_float(h << 16);
}

// A register of two values, of which `own` (a mask of bits) marks those of the round's own entries: of these, what
// is not finite is cleared and reported. The others are attended by every token and stay as they are.
template <bool F16>
__device__ __forceinline__ uint32_t finite2(uint32_t x, uint32_t own, bool& odd) {
  constexpr uint32_t e = F16 ? 0x7c00u : 0x7f80u;
  const uint32_t y = x & own;
  if ((y & e) == e) {
    odd = true;
    x &= 0xffff0000u;
  }
  if (((y >> 16) & e) == e) {
    odd = true;
    x &= 0xffffu;
  }
  return x;
}

// Tokens behind a row's get zeros, rows in error NaN; every thread of the CTA.
__device__ __forceinline__ void fill_unused(const AttendParams& P, int D, int tid, int threads) {
  const Round& R = P.R;
  const int per = P.Hq * D / 8;
  for (int b = blockIdx.x; b < R.B; b += gridDim.x) {
    RowWork w;
    const bool ok = row_work(R, b, &w);
    const int i0 = ok ? w.m : 0;
    const uint32_t v = ok ? 0u : 0x7fff7fffu;                 // NaN in both types
    uint4* o = reinterpret_cast<uint4*>(P.out) + (static_cast<size_t>(b) * R.N + i0) * per;
    for (int x = tid; x < (R.N - i0) * per; x += threads) o[x] = make_uint4(v, v, v, v);
    if (P.lse) {
      float* l = P.lse + (static_cast<size_t>(b) * R.N + i0) * P.Hq;
      for (int x = tid; x < (R.N - i0) * P.Hq; x += threads) l[x] = ok ? 0.0f : __int_as_float(0x7fffffff);
    }
  }
}

// The item that this CTA begins, for the join kernel (one thread).
__device__ __forceinline__ void tell_shared(const AttendParams& P, int way, int row, int head, int q_tile, int rows,
                                            bool whole, long long item_at, int tiles, const Plan& plan) {
  if (whole && !P.by_item) return;
  const int cta = blockIdx.x, last = unit_owner(item_at + tiles - 1, plan);
  if (P.by_item)
    P.shared[(row * P.R.C.heads + head) * P.by_item + q_tile] = make_int4(whole ? -1 : cta, 0, rows, last);
  else
    P.shared[cta * P.ways + way] = make_int4(row, head, q_tile << 8 | rows, last);
}
__device__ __forceinline__ void tell_shared(const SharedParams& P, int row, int head, int q_tile, int tokens, int token0,
                                            bool whole, long long item_at, int tiles, const Plan& plan) {
  P.records[P.record_at(row, head, q_tile, token0)] =
      make_int2(whole ? -1 : static_cast<int>(blockIdx.x), whole ? 0 : unit_owner(item_at + static_cast<long long>(tiles - 1) * P.R.units(tokens), plan));
}

// A launch whose CTAs may begin before the kernel ahead of it in the stream ends (which they wait for themselves).
template <class Kern, class... Args>
inline int launch_ahead(Kern kern, dim3 grid, int threads, size_t shared, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

// Joins the parts of the items that the attention kernel's `grid` CTAs shared.
int launch_attend_join(const AttendParams& P, bool f16, bool wide, int grid, cudaStream_t st);

// The wide kernel (at most 128 query heads a key head; query tiles of tile_rows <= 128 rows, whole tokens of
// which q's boxes hold q_tokens; key tiles of 128, or of 64 for heads of 256; two ways up to heads of 128).
int launch_attend_wide(const AttendParams& P, bool f16, const CUtensorMap& k, const CUtensorMap& v,
                       const CUtensorMap& q, int q_tokens, int grid, cudaStream_t st);
// The same of rows that share fronts (q's boxes run over all of the batch's tokens).
int launch_attend_shared(const SharedParams& P, bool f16, const CUtensorMap& k, const CUtensorMap& v,
                         const CUtensorMap& q, int q_tokens, int grid, cudaStream_t st);

}  // namespace sv
