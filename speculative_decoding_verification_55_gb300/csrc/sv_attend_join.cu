// Join of the parts of attention items that many CTAs share (few rows and heads with long caches).
//
//   out = sum_p 2^(c (m_p - M)) o_p / sum_p 2^(c (m_p - M)) l_p,  M = max_p m_p,  over an item's parts p.
//
// One CTA per item and group of rows: 128 threads take four columns of a row each, and four such sets
// of threads a quarter of the parts, with eight loads in flight each. The last arrival of an item joins
// alone otherwise (sv_attend.cuh): as fast for a few parts and one launch less, but with 76 parts
// of 40 rows it took 30 us, this kernel 4.

#include "sv_attend.cuh"

namespace {

constexpr int kSets = 4, kSetThreads = 128, kThreads = kSets * kSetThreads;
constexpr int kMaxParts = 320;

template <bool F16, int D>
__global__ void __launch_bounds__(kThreads) sv_attend_join_kernel(const sv::AttendParams P, int item_rows) {
  constexpr int kAcross = D / 4, kRowsHere = kSetThreads / kAcross;   // threads of a row; rows of the CTA
  __shared__ float factor[kRowsHere][kMaxParts];
  __shared__ float4 part[kSets - 1][kSetThreads];
  __shared__ float total[kRowsHere];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const sv::Round& R = P.R;
  const int c0 = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int4 it = __ldcg(P.shared + c0);
  if (it.x < 0) return;                                // no shared item begins in this CTA's run
  sv::RowWork w;
  sv::row_work(R, it.x, &w);
  const int row0 = it.z * item_rows, rows = min(item_rows, w.m * R.group - row0);
  const int r0 = blockIdx.y * kRowsHere, parts = it.w - c0 + 1;
  if (r0 >= rows) return;
  const float c = P.c;
  for (int x = warp; x < kRowsHere && r0 + x < rows; x += kThreads / 32) {
    float M = -INFINITY, L = 0.0f;
    for (int p = lane; p < parts; p += 32)
      M = fmaxf(M, __ldcg(&P.part_ml[(2 * (c0 + p) + (p == 0)) * item_rows + r0 + x].x));
    M = sv::warp_max(M);
    for (int p = lane; p < parts; p += 32) {
      const float2 e = __ldcg(P.part_ml + (2 * (c0 + p) + (p == 0)) * item_rows + r0 + x);
      const float f = e.x > -INFINITY ? sv::ex2((e.x - M) * c) : 0.0f;
      factor[x][p] = f;
      L += e.x > -INFINITY ? e.y * f : e.y;            // 0, or NaN
    }
    L = sv::warp_sum_lane0(L);
    if (lane == 0) {
      total[x] = L;
      const int i = (row0 + r0 + x) / R.group, hq = it.y * R.group + (row0 + r0 + x) - i * R.group;
      if (P.lse) P.lse[(static_cast<size_t>(it.x) * R.N + i) * P.Hq + hq] = (M * c + log2f(L)) * 0.6931471805599453f;
    }
  }
  __syncthreads();
  const int set = tid / kSetThreads, s = tid % kSetThreads, x = s / kAcross, col = (s % kAcross) * 4;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (r0 + x < rows) {
#pragma unroll 8
    for (int p = set; p < parts; p += kSets) {
      const float4 e = __ldcg(reinterpret_cast<const float4*>(
          P.part_o + (static_cast<size_t>(2 * (c0 + p) + (p == 0)) * item_rows + r0 + x) * D + col));
      const float f = factor[x][p];
      a.x += e.x * f;
      a.y += e.y * f;
      a.z += e.z * f;
      a.w += e.w * f;
    }
  }
  if (set) part[set - 1][s] = a;
  __syncthreads();
  if (set || r0 + x >= rows) return;
#pragma unroll
  for (int y = 0; y < kSets - 1; ++y) {
    const float4 e = part[y][s];
    a.x += e.x;
    a.y += e.y;
    a.z += e.z;
    a.w += e.w;
  }
  const float inv = 1.0f / total[x];
  const int i = (row0 + r0 + x) / R.group, hq = it.y * R.group + (row0 + r0 + x) - i * R.group;
  uint2 v;
  v.x = sv::pack2<F16>(a.x * inv, a.y * inv);
  v.y = sv::pack2<F16>(a.z * inv, a.w * inv);
  *reinterpret_cast<uint2*>(static_cast<char*>(P.out) + (((static_cast<size_t>(it.x) * R.N + i) * P.Hq + hq) * D + col) * 2) = v;
}

template <bool F16, int D>
int launch(const sv::AttendParams& P, int item_rows, int grid, cudaStream_t st) {
  const int most = min(item_rows, P.R.N * P.R.group), here = kSetThreads / (D / 4);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, (most + here - 1) / here);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sv_attend_join_kernel<F16, D>, P, item_rows) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace

namespace sv {

int launch_attend_join(const AttendParams& P, bool f16, int item_rows, int grid, cudaStream_t st) {
  switch (P.R.C.head_dim) {
    case 64: return f16 ? launch<true, 64>(P, item_rows, grid, st) : launch<false, 64>(P, item_rows, grid, st);
    case 128: return f16 ? launch<true, 128>(P, item_rows, grid, st) : launch<false, 128>(P, item_rows, grid, st);
    default: return f16 ? launch<true, 256>(P, item_rows, grid, st) : launch<false, 256>(P, item_rows, grid, st);
  }
}

}  // namespace sv
