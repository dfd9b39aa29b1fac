// What the two attention kernels share: their arguments and the handling of values that are not finite.
#pragma once

#include "sv_tiles.cuh"

namespace sv {

struct AttendParams {
  Round R;
  const char* q;
  long long row_stride, token_stride;          // bytes
  const int32_t* parents;
  void* out;
  float* lse;
  float c;                                     // scale * log2(e)
  int Hq;
  unsigned* counters;                          // [grid] arrivals at the item whose first part it holds
  float* part_o;                               // [2 grid][rows][D]
  float2* part_ml;                             // [2 grid][rows] maximum and sum
};

template <bool F16>
__device__ __forceinline__ float value_of(uint32_t h) {
  if (F16) return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
  return __uint_as_float(h << 16);
}

// A register of two values with those of entries >= `total` (bit masks keep_lo, keep_hi) cleared, and
// those that are not finite cleared and reported.
template <bool F16>
__device__ __forceinline__ uint32_t finite2(uint32_t x, uint32_t keep, bool& odd) {
  constexpr uint32_t e = F16 ? 0x7c00u : 0x7f80u;
  x &= keep;
  if ((x & e) == e) {
    odd = true;
    x &= 0xffff0000u;
  }
  if (((x >> 16) & e) == e) {
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

// An item of several CTAs, whose parts are in the workspace: the last CTA to arrive joins them. The
// item's first part is part 2 p + 1 of the CTA p that holds its first tile, the others part 2 p of
// theirs. kThreads threads meeting at named barrier 1; fin: 2 kRows floats of shared memory.
template <bool F16, int D, int kRows, int kThreads>
__device__ void join_parts(const AttendParams& P, const Walk& W, const Plan& plan, int row0, int rows,
                           int tid, float* fin, int* sm_last) {
  const Round& R = P.R;
  const float c = P.c;
  const long long item_at = W.at - W.first;
  const int c0 = tile_owner(item_at, plan), c1 = tile_owner(item_at + W.w.tiles - 1, plan);
  named_bar_sync(1, kThreads);
  if (tid == 0) {
    __threadfence();
    const unsigned old = atomicAdd(P.counters + c0, 1u);
    *sm_last = old == static_cast<unsigned>(c1 - c0);
    if (*sm_last) P.counters[c0] = 0u;       // left zero for the next call
    __threadfence();
  }
  named_bar_sync(1, kThreads);
  if (!*sm_last) return;
  for (int r = tid; r < rows; r += kThreads) {   // per row: the maximum and 1 / sum
    float jm = -INFINITY, jl = 0.0f;
#pragma unroll 4
    for (int p = c0; p <= c1; ++p) jm = fmaxf(jm, __ldcg(&P.part_ml[(2 * p + (p == c0)) * kRows + r].x));
#pragma unroll 4
    for (int p = c0; p <= c1; ++p) {
      const float2 e = __ldcg(P.part_ml + (2 * p + (p == c0)) * kRows + r);
      jl += e.x > -INFINITY ? e.y * ex2((e.x - jm) * c) : e.y;
    }
    fin[2 * r] = jm;
    fin[2 * r + 1] = 1.0f / jl;
    const int i = (row0 + r) / R.group, hq = W.head * R.group + (row0 + r) - i * R.group;
    if (P.lse) P.lse[(static_cast<size_t>(W.row) * R.N + i) * P.Hq + hq] = (jm * c + log2f(jl)) * 0.6931471805599453f;
  }
  named_bar_sync(1, kThreads);
  for (int x = tid; x < rows * (D / 4); x += kThreads) {
    const int r = x / (D / 4), col = (x % (D / 4)) * 4;
    const float jm = fin[2 * r], inv = fin[2 * r + 1];
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int p = c0; p <= c1; ++p) {
      const int sl = 2 * p + (p == c0);
      const float pm = __ldcg(&P.part_ml[sl * kRows + r].x);
      const float4 e = __ldcg(reinterpret_cast<const float4*>(P.part_o + (static_cast<size_t>(sl) * kRows + r) * D + col));
      const float f = pm == -INFINITY ? 0.0f : ex2((pm - jm) * c);
      a.x += e.x * f;
      a.y += e.y * f;
      a.z += e.z * f;
      a.w += e.w * f;
    }
    const int i = (row0 + r) / R.group, hq = W.head * R.group + (row0 + r) - i * R.group;
    uint2 v;
    v.x = pack2<F16>(a.x * inv, a.y * inv);
    v.y = pack2<F16>(a.z * inv, a.w * inv);
    *reinterpret_cast<uint2*>(static_cast<char*>(P.out) + (((static_cast<size_t>(W.row) * R.N + i) * P.Hq + hq) * D + col) * 2) = v;
  }
  named_bar_sync(1, kThreads);
}

// The wide kernel (64 or 128 elements a head; query rows and tiles of 128).
int launch_attend_wide(const AttendParams& P, bool f16, const CUtensorMap& k, const CUtensorMap& v, int grid,
                       cudaStream_t st);

}  // namespace sv
