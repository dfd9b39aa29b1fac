// Shaping of a round's logits before they are verified, and the token counts that it reads ([R] "Speculative
// decoding", rayaq.ca ml-models -- Why the output is exactly the target's: temperature, top-p and any penalties are
// applied to p and q before the test).
//
//   n = occurrences of token t in the row's output + among the round's tokens that position i follows,
//   z' = z / rep where z > 0, else z * rep, if n > 0 or t is in the prompt (else z);
//   z'' = z' - freq n - pres [n > 0] + sum of t's biases;  -inf where the mask bars t.
//
// In place, one pass, one launch. A thread owns 8 neighbouring tokens of a row (16 bytes of counts, a byte of a mask,
// 16 or 32 bytes of logits) at all of the round's positions: the counts are read once a row, and no two threads share
// a logit. Logits are read only where something changes them, and written only where something does: a group of 8 that
// a mask bars is written without being read.
// Bound: the writes of barred logits, or the reads of the counts where there is no mask.
// Rounding: fp32 throughout, one rounding to the logits' type at the end. Logits that nothing changes keep their bits.

#include <cuda_bf16.h>

#include "sv_cache.cuh"
#include "sv_tiles.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBias = 1024, kMaxRound = SV_MAX_GAMMA + 1;

struct ShapeParams {
  void* logits;
  const int32_t* num;
  const int32_t* tokens;
  const int32_t* parents;
  const int16_t* counts;
  const float* rep;
  const float* freq;
  const float* pres;
  const int32_t* bias_tokens;
  const float* bias;
  const uint8_t* mask;
  long long mask_row, mask_position;           // bytes
  int T, K, N, V, chunks;
  bool penalties;
};

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// kW logits or counts of a thread, moved in words of up to 16 bytes.
template <typename T, int kW>
struct alignas(sizeof(T) * kW < 16 ? sizeof(T) * kW : 16) Group {
  T x[kW];
};

// The round's tokens or the row's biases that fall into a CTA's tokens, in their order; one warp.
__device__ __forceinline__ int gather(const int32_t* from, int n, int v0, int v1, int lane, int* token, int* index,
                                      unsigned* special, int width_log2) {
  int have = 0;
  for (int x0 = 0; x0 < n; x0 += 32) {
    const int t = x0 + lane < n ? __ldg(from + x0 + lane) : -1;
    const bool in = t >= v0 && t < v1;         // (v0 >= 0: a token below 0 is in no CTA's)
    const unsigned all = __ballot_sync(sv::kFull, in);
    if (in) {
      const int at = have + __popc(all & ((1u << lane) - 1));
      token[at] = t;
      index[at] = x0 + lane;
      const int g = (t - v0) >> width_log2;
      atomicOr(special + (g >> 5), 1u << (g & 31));
    }
    have += __popc(all);
  }
  return have;
}

// kW: tokens of a thread, 8 or (rows that are not of whole 16-byte words) 1; kU: groups of a thread.
template <typename T, int kW, int kU>
__global__ void __launch_bounds__(kThreads) sv_shape_kernel(const ShapeParams P) {
  using G = Group<T, kW>;
  constexpr int kSpan = kThreads * kW * kU;    // tokens of a CTA
  constexpr int kLog2 = kW == 8 ? 3 : 0;
  constexpr unsigned kAll = (1u << kW) - 1;
  __shared__ unsigned special[kThreads * kU / 32];
  __shared__ int said[kMaxRound], said_at[kMaxRound], lists[2];
  __shared__ int biased[kMaxBias], biased_at[kMaxBias];
  __shared__ unsigned long long above[sv::kMaxTreeNodes];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / P.chunks, v0 = (blockIdx.x - b * P.chunks) * kSpan, v1 = min(v0 + kSpan, P.V);
  const int m = P.num ? __ldg(P.num + b) : P.N;

  // Counts first: they take the longest to come.
  Group<int16_t, kW> n0[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int v = v0 + (u * kThreads + tid) * kW;
#pragma unroll
    for (int k = 0; k < kW; ++k) n0[u].x[k] = 0;
    if (P.counts && v < v1)
      n0[u] = *reinterpret_cast<const Group<int16_t, kW>*>(P.counts + static_cast<size_t>(b) * P.V + v);
  }
  for (int x = tid; x < kThreads * kU / 32; x += kThreads) special[x] = 0;
  bool ok = m >= 0 && m <= P.N;
  if (ok && P.parents) ok = sv::tree_masks(P.parents + static_cast<size_t>(b) * P.N, m, above, tid, kThreads);
  if (!__syncthreads_and(ok) || m == 0) return;
  // A chain's position i follows tokens 0 .. i - 1, a tree's node i follows its ancestors and itself.
  if (warp == 0) {
    const int have = P.tokens && P.penalties
                         ? gather(P.tokens + static_cast<size_t>(b) * P.T, P.parents ? m : m - 1, v0, v1, lane, said, said_at, special, kLog2)
                         : 0;
    if (lane == 0) lists[0] = have;
  } else if (warp == 1) {
    const int have = gather(P.bias_tokens + static_cast<size_t>(b) * P.K, P.K, v0, v1, lane, biased, biased_at, special, kLog2);
    if (lane == 0) lists[1] = have;
  }
  const float rep = P.rep ? __ldg(P.rep + b) : 1.0f, freq = P.freq ? __ldg(P.freq + b) : 0.0f;
  const float pres = P.pres ? __ldg(P.pres + b) : 0.0f;
  __syncthreads();

  const uint8_t* const mask = P.mask ? P.mask + b * P.mask_row : nullptr;
  T* const row = static_cast<T*>(P.logits) + static_cast<size_t>(b) * P.N * P.V;
  const float inf = __int_as_float(0x7f800000);
#pragma unroll 1
  for (int u = 0; u < kU; ++u) {
    const int g = u * kThreads + tid, v = v0 + g * kW;
    if (v >= v1) break;
    const bool odd = (special[g >> 5] >> (g & 31)) & 1;
    bool any = odd;
#pragma unroll
    for (int k = 0; k < kW; ++k) any |= n0[u].x[k] != 0;
    if (!any && !mask) continue;
    float add[kW];
    unsigned touched = 0;
#pragma unroll
    for (int k = 0; k < kW; ++k) add[k] = 0.0f;
    if (odd)
      for (int e = 0; e < lists[1]; ++e) {
        const float f = __ldg(P.bias + static_cast<size_t>(b) * P.K + biased_at[e]);
#pragma unroll
        for (int k = 0; k < kW; ++k)
          if (biased[e] == v + k) {
            add[k] += f;
            touched |= 1u << k;
          }
      }
    constexpr int kBatch = 4;                  // positions whose loads are in flight together
    for (int i0 = 0; i0 < m; i0 += kBatch) {
      unsigned allowed[kBatch];
      G z[kBatch];
#pragma unroll
      for (int y = 0; y < kBatch; ++y) {
        allowed[y] = kAll;
        if (mask && i0 + y < m) allowed[y] = __ldg(mask + (i0 + y) * P.mask_position + (v >> 3)) >> (kW == 8 ? 0 : v & 7) & kAll;
      }
#pragma unroll
      for (int y = 0; y < kBatch; ++y)
        if (i0 + y < m && allowed[y] && (any || allowed[y] != kAll))
          z[y] = *reinterpret_cast<const G*>(row + static_cast<size_t>(i0 + y) * P.V + v);
#pragma unroll
      for (int y = 0; y < kBatch; ++y) {
        const int i = i0 + y;
        if (i >= m || (!any && allowed[y] == kAll)) continue;
        if (any && allowed[y]) {
          int n[kW];
#pragma unroll
          for (int k = 0; k < kW; ++k) n[k] = n0[u].x[k] & 32767;
          if (odd)
            for (int e = 0; e < lists[0]; ++e) {
              const int a = said_at[e];        // (place 0 of a tree, the root, is above every node)
              const bool follows = P.parents ? a == 0 || ((above[i] >> (a - 1)) & 1) : a < i;
#pragma unroll
              for (int k = 0; k < kW; ++k) n[k] += follows && said[e] == v + k;
            }
#pragma unroll
          for (int k = 0; k < kW; ++k) {
            const bool seen = n[k] > 0 || n0[u].x[k] < 0;
            if (!seen && !((touched >> k) & 1)) continue;
            float x = to_float<T>(z[y].x[k]);
            if (seen) x = x > 0.0f ? x / rep : x * rep;
            x -= freq * static_cast<float>(n[k]);
            if (n[k] > 0) x -= pres;
            z[y].x[k] = from_float<T>(x + add[k]);
          }
        }
#pragma unroll
        for (int k = 0; k < kW; ++k)
          if (!((allowed[y] >> k) & 1)) z[y].x[k] = from_float<T>(-inf);
        *reinterpret_cast<G*>(row + static_cast<size_t>(i) * P.V + v) = z[y];
      }
    }
  }
}

template <typename T>
int launch_shape(ShapeParams& P, int B, bool whole, int sms, cudaStream_t st) {
  // Four groups a thread where that still leaves eight CTAs an SM, else one.
  const long long groups = static_cast<long long>(B) * ((P.V + 7) / 8);
  const bool four = groups / (4 * kThreads) >= 8ll * sms;
  const int span = kThreads * (whole ? (four ? 32 : 8) : 8);
  P.chunks = (P.V + span - 1) / span;
  const long long grid = static_cast<long long>(B) * P.chunks;
  if (grid > 0x7fffffffll) return SV_ERR_BAD_SHAPE;
  if (!whole) sv_shape_kernel<T, 1, 8><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(P);
  else if (four) sv_shape_kernel<T, 8, 4><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(P);
  else sv_shape_kernel<T, 8, 1><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(P);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

// ------------------------------------------------------------------------------------------------
// Token counts
// ------------------------------------------------------------------------------------------------

constexpr int kPer = 4;                        // tokens of a thread

// Occurrences of a token among a warp's lanes are added once, by the first of them. The sum and its limit do not
// depend on the order in which threads come.
__global__ void __launch_bounds__(kThreads) sv_count_kernel(const int32_t* tokens, const int32_t* num, int16_t* counts,
                                                            int M, int V, int chunks, bool prompt) {
  const int b = blockIdx.x / chunks, x0 = (blockIdx.x - b * chunks) * (kThreads * kPer);
  const int m = num ? __ldg(num + b) : M;
  if (m > M || x0 >= m) return;
  unsigned short* const row = reinterpret_cast<unsigned short*>(counts) + static_cast<size_t>(b) * V;
  int t[kPer];
#pragma unroll
  for (int y = 0; y < kPer; ++y) {
    const int x = x0 + y * kThreads + threadIdx.x;
    t[y] = x < m ? __ldg(tokens + static_cast<size_t>(b) * M + x) : -1;
    if (static_cast<unsigned>(t[y]) >= static_cast<unsigned>(V)) t[y] = -1;
  }
  if (prompt) {
    unsigned short c[kPer];
#pragma unroll
    for (int y = 0; y < kPer; ++y) c[y] = t[y] >= 0 ? __ldcg(row + t[y]) : 0x8000;
#pragma unroll
    for (int y = 0; y < kPer; ++y)             // whoever writes a token in this call writes the same
      if (!(c[y] & 0x8000)) __stcg(row + t[y], static_cast<unsigned short>(c[y] | 0x8000));
    return;
  }
#pragma unroll
  for (int y = 0; y < kPer; ++y) {
    const unsigned same = __match_any_sync(sv::kFull, t[y]);
    if (t[y] < 0 || (threadIdx.x & 31) != __ffs(same) - 1) continue;
    const int n = __popc(same);
    unsigned short* const at = row + t[y];
    unsigned short old = __ldcg(at);
    for (;;) {                                 // ends: another thread's addition is what makes a turn fail
      const int sum = min((old & 32767) + n, 32767);
      const unsigned short now = atomicCAS(at, old, static_cast<unsigned short>((old & 0x8000) | sum));
      if (now == old) break;
      old = now;
    }
  }
}

}  // namespace

extern "C" int spec_verify_shape_logits(void* logits, const int32_t* num_positions, const int32_t* tokens, int32_t T,
                                        const int32_t* tree_parents, const int16_t* counts, const float* repetition,
                                        const float* frequency, const float* presence, const int32_t* bias_tokens,
                                        const float* bias, int32_t K, const int32_t* mask, int32_t mask_positions,
                                        int32_t B, int32_t N, int32_t V, int32_t dtype, void* cuda_stream) {
  if (dtype != SV_DTYPE_F32 && dtype != SV_DTYPE_BF16) return SV_ERR_BAD_DTYPE;
  if (!logits || (bias_tokens == nullptr) != (bias == nullptr) || (tree_parents && !tokens)) return SV_ERR_NULL_POINTER;
  if (B < 1 || B > (1 << 20) || N < 1 || N > kMaxRound || V < 1 || V > (1 << 24)) return SV_ERR_BAD_SHAPE;
  if (tokens && (T < (tree_parents ? N : N - 1) || T > (1 << 20))) return SV_ERR_BAD_SHAPE;
  if (bias && (K < 0 || K > kMaxBias)) return SV_ERR_BAD_SHAPE;
  if (mask && mask_positions != N && mask_positions != 1) return SV_ERR_BAD_SHAPE;
  const int size = dtype == SV_DTYPE_F32 ? 4 : 2;
  if (sv::misaligned(logits, size) || sv::misaligned(counts, 2)) return SV_ERR_MISALIGNED;
  for (const void* p : {static_cast<const void*>(num_positions), static_cast<const void*>(tokens),
                        static_cast<const void*>(tree_parents), static_cast<const void*>(repetition),
                        static_cast<const void*>(frequency), static_cast<const void*>(presence),
                        static_cast<const void*>(bias_tokens), static_cast<const void*>(bias), static_cast<const void*>(mask)})
    if (sv::misaligned(p, 4)) return SV_ERR_MISALIGNED;
  const unsigned long long rows = B, words = (V + 31) / 32;
  if (sv::overlap({{logits, rows * N * V * size}},
                  {{num_positions, 4 * rows}, {tokens, 4 * rows * (tokens ? T : 0)}, {tree_parents, 4 * rows * N},
                   {counts, 2 * rows * V}, {repetition, 4 * rows}, {frequency, 4 * rows}, {presence, 4 * rows},
                   {bias_tokens, 4 * rows * (bias ? K : 0)}, {bias, 4 * rows * (bias ? K : 0)},
                   {mask, 4 * rows * words * (mask ? mask_positions : 0)}}))
    return SV_ERR_OVERLAP;
  int dev = 0;
  const int st = sv::current_device_status(&dev);
  if (st != SV_OK) return st;
  const int sms = sv::device_sms(dev);
  if (sms < 1) return SV_ERR_CUDA;
  ShapeParams P;
  P.logits = logits;
  P.num = num_positions;
  P.tokens = tokens;
  P.parents = tree_parents;
  P.penalties = repetition || frequency || presence;
  P.counts = P.penalties ? counts : nullptr;
  P.rep = repetition;
  P.freq = frequency;
  P.pres = presence;
  P.bias_tokens = bias_tokens;
  P.bias = bias;
  P.mask = reinterpret_cast<const uint8_t*>(mask);
  P.mask_row = static_cast<long long>(4 * words) * mask_positions;
  P.mask_position = mask_positions == 1 ? 0 : static_cast<long long>(4 * words);
  P.T = T;
  P.K = bias ? K : 0;
  P.N = N;
  P.V = V;
  if (!P.penalties && P.K == 0 && !mask) return SV_OK;
  // Whole 16-byte words of counts are whole ones of logits too.
  const bool whole = V % 8 == 0 && !sv::misaligned(logits, 16) && !sv::misaligned(P.counts, 16);
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  return dtype == SV_DTYPE_F32 ? launch_shape<float>(P, B, whole, sms, s) : launch_shape<__nv_bfloat16>(P, B, whole, sms, s);
}

extern "C" int spec_verify_count_tokens(const int32_t* tokens, const int32_t* num, int16_t* counts, int32_t prompt,
                                        int32_t B, int32_t M, int32_t V, void* cuda_stream) {
  if (!tokens || !counts) return SV_ERR_NULL_POINTER;
  if (B < 1 || B > (1 << 20) || M < 1 || V < 1 || V > (1 << 24)) return SV_ERR_BAD_SHAPE;
  const int chunks = (M - 1) / (kThreads * kPer) + 1;
  if (static_cast<long long>(B) * chunks > 0x7fffffffll) return SV_ERR_BAD_SHAPE;
  if (sv::misaligned(tokens, 4) || sv::misaligned(num, 4) || sv::misaligned(counts, 2)) return SV_ERR_MISALIGNED;
  const unsigned long long rows = B;
  if (sv::overlap({{counts, 2 * rows * V}}, {{tokens, 4 * rows * M}, {num, 4 * rows}})) return SV_ERR_OVERLAP;
  int dev = 0;
  const int st = sv::current_device_status(&dev);
  if (st != SV_OK) return st;
  sv_count_kernel<<<B * chunks, kThreads, 0, static_cast<cudaStream_t>(cuda_stream)>>>(tokens, num, counts, M, V, chunks,
                                                                                     prompt != 0);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
