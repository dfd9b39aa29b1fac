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
  int4* shared;                                // [grid] that item, for the join kernel (null: the last
                                               // arrival joins): row, head, query tile, its last CTA
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

// An item of several CTAs, whose parts are in the workspace: the last CTA to arrive joins them, or the
// join kernel does. The item's first part is part 2 p + 1 of the CTA p that holds its first tile, the
// others part 2 p of theirs. kThreads threads meeting at named barrier 1; fin: 2 kRows floats of shared
// memory.
template <bool F16, int D, int kRows, int kThreads>
__device__ void join_parts(const AttendParams& P, const Walk& W, const Plan& plan, int row0, int rows,
                           int tid, float* fin, int* sm_last) {
  const Round& R = P.R;
  const float c = P.c;
  const int c0 = unit_owner(W.item_at, plan), c1 = unit_owner(W.item_at + W.w.tiles - 1, plan);
  if (P.shared) {
    if (tid == 0 && W.first == 0) P.shared[blockIdx.x] = make_int4(W.row, W.head, W.q_tile, c1);
    named_bar_sync(1, kThreads);             // the shared memory is free for the next item
    return;
  }
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
  for (int r = tid >> 5; r < rows; r += kThreads / 32) {   // per row: the maximum and 1 / sum
    float jm = -INFINITY, jl = 0.0f;
    for (int p = c0 + (tid & 31); p <= c1; p += 32)
      jm = fmaxf(jm, __ldcg(&P.part_ml[(2 * p + (p == c0)) * kRows + r].x));
    jm = warp_max(jm);
    for (int p = c0 + (tid & 31); p <= c1; p += 32) {
      const float2 e = __ldcg(P.part_ml + (2 * p + (p == c0)) * kRows + r);
      jl += e.x > -INFINITY ? e.y * ex2((e.x - jm) * c) : e.y;
    }
    jl = warp_sum_lane0(jl);
    if ((tid & 31) == 0) {
      fin[2 * r] = jm;
      fin[2 * r + 1] = 1.0f / jl;
      const int i = (row0 + r) / R.group, hq = W.head * R.group + (row0 + r) - i * R.group;
      if (P.lse) P.lse[(static_cast<size_t>(W.row) * R.N + i) * P.Hq + hq] = (jm * c + log2f(jl)) * 0.6931471805599453f;
    }
  }
  named_bar_sync(1, kThreads);
  // Four columns of kAcross rows a thread at a time, and two parts of each: loads of that many parts in
  // flight.
  constexpr int kAcross = kRows >= 64 ? 4 : 2, kStep = kThreads / (D / 4);
  const int col = (tid % (D / 4)) * 4;
  for (int r0 = tid / (D / 4); r0 < rows; r0 += kAcross * kStep) {
    float4 a[kAcross];
    float jm[kAcross];
#pragma unroll
    for (int x = 0; x < kAcross; ++x) {
      a[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      jm[x] = fin[2 * min(r0 + x * kStep, rows - 1)];
    }
#pragma unroll 2
    for (int p = c0; p <= c1; ++p) {
      const int sl = 2 * p + (p == c0);
      float pm[kAcross];
      float4 e[kAcross];
#pragma unroll
      for (int x = 0; x < kAcross; ++x) {
        const size_t at = static_cast<size_t>(sl) * kRows + min(r0 + x * kStep, rows - 1);
        pm[x] = __ldcg(&P.part_ml[at].x);
        e[x] = __ldcg(reinterpret_cast<const float4*>(P.part_o + at * D + col));
      }
#pragma unroll
      for (int x = 0; x < kAcross; ++x) {
        const float f = pm[x] == -INFINITY ? 0.0f : ex2((pm[x] - jm[x]) * c);
        a[x].x += e[x].x * f;
        a[x].y += e[x].y * f;
        a[x].z += e[x].z * f;
        a[x].w += e[x].w * f;
      }
    }
#pragma unroll
    for (int x = 0; x < kAcross; ++x) {
      const int r = r0 + x * kStep;
      if (r >= rows) break;
      const float inv = fin[2 * r + 1];
      const int i = (row0 + r) / R.group, hq = W.head * R.group + (row0 + r) - i * R.group;
      uint2 v;
      v.x = pack2<F16>(a[x].x * inv, a[x].y * inv);
      v.y = pack2<F16>(a[x].z * inv, a[x].w * inv);
      *reinterpret_cast<uint2*>(static_cast<char*>(P.out) + (((static_cast<size_t>(W.row) * R.N + i) * P.Hq + hq) * D + col) * 2) = v;
    }
  }
  named_bar_sync(1, kThreads);
}

// Joins the parts of the items that main kernel's CTAs shared (P.shared), rows of `item_rows` each.
int launch_attend_join(const AttendParams& P, bool f16, int item_rows, int grid, cudaStream_t st);

// The wide kernel (64 or 128 elements a head; query rows and tiles of 128).
int launch_attend_wide(const AttendParams& P, bool f16, const CUtensorMap& k, const CUtensorMap& v, int grid,
                       cudaStream_t st);

}  // namespace sv
