// Join of the parts of attention items that several CTAs shared.
//
//   out = sum_p 2^(c (m_p - M)) o_p / sum_p 2^(c (m_p - M)) l_p,  M = max_p m_p,  over an item's parts p.
//
// A part is o [D][rows] and (m, l) [rows] in fp32: a lane has a row (and reads whole lines with its
// neighbours) and 8 or 16 columns. 16 warps a CTA divide its columns and the parts among them, each with a
// running maximum over its parts, and meet in shared memory. With few items, which then have many
// parts, a CTA takes 8 columns of an item (16 of a tile of 16 rows) and each warp a sixteenth of the parts, a CTA a
// possible item and not a CTA of the attention's; otherwise all columns.
// Every item that is not whole goes through here. Joining in the last CTA to arrive instead kept that
// CTA 10 us (3 parts of 128 rows) to 30 us (76 parts of 40 rows); this kernel is launched ahead (its
// CTAs wait for the attention's end) and takes 2 to 4.

#include "sv_attend.cuh"

namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;

template <bool F16, int D, int kRows, int kAcross, int kCols>    // kAcross: warps across the columns
__global__ void __launch_bounds__(kThreads) sv_attend_join_kernel(const sv::AttendParams P) {
  constexpr int kRowLanes = kRows < 32 ? kRows : 32, kColLanes = 32 / kRowLanes;
  constexpr int kPartGroups = kWarps / kAcross, kColsHere = kAcross * kColLanes * kCols;
  constexpr int kColBlocks = D / kColsHere;
  __shared__ float acc[kWarps][kCols][33];
  __shared__ float2 ml[kWarps][32];
  const sv::Round& R = P.R;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int4 it;                                             // row, head, query tile, the last CTA
  int c0, way, rows;
  if (kCols == 8) {                                    // records by item; the lengths were there before the attention
    const int id = blockIdx.x, pair = id / P.by_item;
    it = make_int4(pair / R.C.heads, pair % R.C.heads, id % P.by_item, 0);
    way = it.z % P.ways;
    sv::RowWork w;
    sv::row_work(R, it.x, &w);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (w.q_tiles == 0 || it.z * P.tile_rows >= w.m * R.group) return;
    const int4 e = __ldcg(P.shared + id);
    if (e.x < 0) return;                               // a CTA had all of it
    c0 = e.x;
    rows = e.z;
    it.w = e.w;
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    it = __ldcg(P.shared + blockIdx.x);
    if (it.x < 0) return;                              // no shared item begins in this CTA's run
    c0 = blockIdx.x / P.ways;
    way = blockIdx.x % P.ways;
    rows = it.z & 255;
    it.z >>= 8;
  }
  const int row0 = it.z * P.tile_rows;
  const int g0 = (blockIdx.y / kColBlocks) * kRowLanes, col0 = (blockIdx.y % kColBlocks) * kColsHere;
  if (g0 >= rows) return;
  const float c = P.c;
  {
    const int r = g0 + lane % kRowLanes, pg = warp / kAcross;
    const int col = col0 + ((warp % kAcross) * kColLanes + lane / kRowLanes) * kCols;
    float M = -INFINITY, L = 0.0f, a[kCols];
#pragma unroll
    for (int x = 0; x < kCols; ++x) a[x] = 0.0f;
#pragma unroll(kCols == 8 ? 4 : 2)
    for (int p = c0 + pg; p <= it.w; p += kPartGroups) {
      const size_t part = static_cast<size_t>(2 * p + (p == c0)) * P.ways + way;
      const float2 e = __ldcg(P.part_ml + part * kRows + r);
      float o[kCols];
#pragma unroll
      for (int x = 0; x < kCols; ++x) o[x] = __ldcg(P.part_o + (part * D + col + x) * kRows + r);
      const float top = fmaxf(M, e.x);
      const float f = M == top ? 1.0f : (M == -INFINITY ? 0.0f : sv::ex2((M - top) * c));
      const float g = e.x == -INFINITY ? 0.0f : sv::ex2((e.x - top) * c);
      M = top;
      L = L * f + (e.x == -INFINITY ? e.y : e.y * g);  // the former: 0, or NaN
#pragma unroll
      for (int x = 0; x < kCols; ++x) a[x] = a[x] * f + o[x] * g;   // (an infinity times a weight of 0: NaN)
    }
#pragma unroll
    for (int x = 0; x < kCols; ++x) acc[warp][x][lane] = a[x];
    ml[warp][lane] = make_float2(M, L);
  }
  __syncthreads();
  // kAcross columns of a row a thread.
  constexpr int kChunks = kColsHere / kAcross;
  const int r = tid / kChunks, first = (tid % kChunks) * kAcross;
  if (r >= kRowLanes || g0 + r >= rows) return;
  float M = -INFINITY, L = 0.0f, f[kPartGroups], v[kAcross];
#pragma unroll
  for (int g = 0; g < kPartGroups; ++g) M = fmaxf(M, ml[g * kAcross][r].x);
#pragma unroll
  for (int g = 0; g < kPartGroups; ++g) {
    const float2 e = ml[g * kAcross][r];
    f[g] = e.x == -INFINITY ? 0.0f : sv::ex2((e.x - M) * c);
    L += e.x == -INFINITY ? e.y : e.y * f[g];
  }
  const float inv = 1.0f / L;
  const int i = (row0 + g0 + r) / R.group, hq = it.y * R.group + (row0 + g0 + r) - i * R.group;
  const size_t at = (static_cast<size_t>(it.x) * R.N + i) * P.Hq + hq;
#pragma unroll
  for (int x = 0; x < kAcross; ++x) {
    const int col = first + x, wc = col / (kColLanes * kCols), cl = (col / kCols) % kColLanes;
    float s = 0.0f;
#pragma unroll
    for (int g = 0; g < kPartGroups; ++g) s += acc[g * kAcross + wc][col % kCols][cl * kRowLanes + r] * f[g];
    v[x] = s * inv;
  }
  char* out = static_cast<char*>(P.out) + (at * D + col0 + first) * 2;
  if constexpr (kAcross == 1) {
    if (F16) *reinterpret_cast<__half*>(out) = __float2half_rn(v[0]);
    else *reinterpret_cast<__nv_bfloat16*>(out) = __float2bfloat16_rn(v[0]);
  } else {
#pragma unroll
    for (int x = 0; x < kAcross; x += 2) reinterpret_cast<uint32_t*>(out)[x / 2] = sv::pack2<F16>(v[x], v[x + 1]);
  }
  if (P.lse && col0 + first == 0) P.lse[at] = (M * c + (log2f(L) - sv::kProbBits<F16, kRows == 128>)) * 0.6931471805599453f;
}

template <bool F16, int D, int kRows, int kAcross, int kCols>
int launch2(const sv::AttendParams& P, int blocks, cudaStream_t st) {
  constexpr int kRowLanes = kRows < 32 ? kRows : 32, kColsHere = kAcross * (32 / kRowLanes) * kCols;
  const int most = min(kRows, P.R.N * P.R.group);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, (most + kRowLanes - 1) / kRowLanes * (D / kColsHere));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sv_attend_join_kernel<F16, D, kRows, kAcross, kCols>, P) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

template <bool F16, int D, int kRows>
int launch(const sv::AttendParams& P, int grid, cudaStream_t st) {
  constexpr int kAll = D / 16 / (kRows < 32 ? 32 / kRows : 1);
  return P.by_item ? launch2<F16, D, kRows, 1, 8>(P, P.R.B * P.R.C.heads * P.by_item, st)
                   : launch2<F16, D, kRows, kAll, 16>(P, grid * P.ways, st);
}

}  // namespace

namespace sv {

int launch_attend_join(const AttendParams& P, bool f16, bool wide, int grid,
                       cudaStream_t st) {
  switch (P.R.C.head_dim) {
    case 64:
      if (wide) return f16 ? launch<true, 64, 128>(P, grid, st) : launch<false, 64, 128>(P, grid, st);
      return f16 ? launch<true, 64, 16>(P, grid, st) : launch<false, 64, 16>(P, grid, st);
    case 128:
      if (wide) return f16 ? launch<true, 128, 128>(P, grid, st) : launch<false, 128, 128>(P, grid, st);
      return f16 ? launch<true, 128, 16>(P, grid, st) : launch<false, 128, 16>(P, grid, st);
    default:
      if (wide) return f16 ? launch<true, 256, 128>(P, grid, st) : launch<false, 256, 128>(P, grid, st);
      return f16 ? launch<true, 256, 16>(P, grid, st) : launch<false, 256, 16>(P, grid, st);
  }
}

}  // namespace sv
