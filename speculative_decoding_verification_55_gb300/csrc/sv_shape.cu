// Shaping of a round's logits before they are verified, and the token counts that it reads ([R] "Speculative
// decoding", rayaq.ca ml-models -- Why the output is exactly the target's: temperature, top-p and any penalties are
// applied to p and q before the test).
//
//   n = occurrences of token t in the row's output + among the round's tokens that position i follows,
//   z' = z / rep where z > 0, else z * rep, if n > 0 or t is in the prompt (else z);
//   z'' = z' - freq n - pres [n > 0] + sum of t's biases;  -inf where the mask bars t.
//
// In place, one launch. A CTA owns a run of a row's tokens at all of the round's positions, in two passes. First, 8
// neighbouring tokens a thread (16 bytes of counts, a byte of a mask, 16 or 32 bytes of logits): the tokens that
// penalties or biases concern go into a list, and what the masks bar is written, groups barred whole without being
// read. Then the list's tokens at each position, one a lane. (Worked on in the first pass, where a warp's 256 tokens
// hold one or two of them, they cost 269 us for 256 rows of 8 x 152064 fp32, bound by the instructions of idle lanes.)
// Bound: the writes of barred logits; else the reads of the counts and the sectors of the logits that change.
// Rounding: fp32 throughout, one rounding to the logits' type at the end. Logits that nothing changes keep their bits.

#include <cuda_bf16.h>

#include "sv_cache.cuh"
#include "sv_tiles.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBias = 1024, kMaxRound = SV_MAX_GAMMA + 1;
constexpr int kPositions = 9;                  // of a CTA at most: a round of eight drafts

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
  const int32_t* mask;
  long long mask_row, mask_position;           // words
  int B, T, K, N, V, blocks, per;              // blocks of `per` positions
  bool penalties, mask_whole;                  // mask rows of whole 16-byte words
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

// kW logits or counts of a thread, moved in words of up to 32 bytes.
template <typename T, int kW>
struct alignas(sizeof(T) * kW) Group {
  T x[kW];
};
template <typename T, int kW>
__device__ __forceinline__ void put(void* at, const Group<T, kW>& g) {
  if constexpr (sizeof(g) == 32) {             // (two words of 16 bytes would each fill half of what a warp's store touches)
    const uint32_t* const w = reinterpret_cast<const uint32_t*>(g.x);
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
  } else {
    *static_cast<Group<T, kW>*>(at) = g;
  }
}

// The round's tokens or the row's biases that fall into a CTA's tokens, in their order; one warp. `next`: the lane's
// among the first 32.
__device__ __forceinline__ int gather(const int32_t* from, int next, int n, int v0, int v1, int lane, int* token,
                                      unsigned short* index, unsigned* special) {
  int have = 0;
  for (int x0 = 0; x0 < n; x0 += 32) {
    const int t = x0 + lane < n ? next : -1;
    next = x0 + 32 + lane < n ? __ldg(from + x0 + 32 + lane) : -1;
    const bool in = t >= v0 && t < v1;         // (v0 >= 0: a token below 0 is in no CTA's)
    const unsigned all = __ballot_sync(sv::kFull, in);
    if (in) {
      const int at = have + __popc(all & ((1u << lane) - 1));
      token[at] = t - v0;
      index[at] = static_cast<unsigned short>(x0 + lane);
      atomicOr(special + ((t - v0) >> 5), 1u << ((t - v0) & 31));
    }
    have += __popc(all);
  }
  return have;
}

// A token of the list: its place in the CTA's run, whether the round's tokens or the biases have it, its count.
constexpr int kPlaceBits = 13;
constexpr unsigned kSpecial = 1u << kPlaceBits;
__device__ __forceinline__ unsigned listed(int place, bool special, int16_t count) {
  return static_cast<unsigned>(place) | (special ? kSpecial : 0u) | static_cast<unsigned>(static_cast<unsigned short>(count)) << 16;
}

// kW: tokens of a thread, 8 or (rows that are not of whole words) 1; kU: groups of a thread.
template <typename T, int kW, int kU>
__global__ void __launch_bounds__(kThreads, 6) sv_shape_kernel(const ShapeParams P) {
  using G = Group<T, kW>;
  constexpr int kSpan = kThreads * kW * kU;    // tokens of a CTA
  constexpr unsigned kAll = (1u << kW) - 1;
  static_assert(kSpan <= 1 << kPlaceBits, "a place in the list");
  __shared__ unsigned special[kSpan / 32];     // a bit a token
  __shared__ __align__(16) unsigned masks[kPositions][kSpan / 32];
  __shared__ unsigned list[kSpan];
  __shared__ int said[kMaxRound], biased[kMaxBias], up[kMaxRound], lists[2], length;
  __shared__ unsigned short said_at[kMaxRound], biased_at[kMaxBias];
  __shared__ unsigned long long above[sv::kMaxTreeNodes];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = blockIdx.x / P.blocks;       // the rows' first runs first: a text's tokens have low numbers
  const int b = run % P.B, v0 = run / P.B * kSpan, v1 = min(v0 + kSpan, P.V);
  const int first = (blockIdx.x - run * P.blocks) * P.per, most = min(P.per, P.N - first);

  // What takes long to come is asked for at once: the row's positions, its masks, its counts, its tree.
  const int m = P.num ? __ldg(P.num + b) : P.N;
  constexpr int kWords = kSpan / 32;           // of a mask
  if (P.mask) {
    const int words = (v1 - v0 + 31) >> 5;
    const int32_t* const from = P.mask + b * P.mask_row + (v0 >> 5);
    for (int y = warp; y < most; y += kThreads / 32) {
      const int32_t* const f = from + (first + y) * P.mask_position;
      const uint32_t to = sv::smem_addr(masks[y]);
      if (P.mask_whole) {
        for (int w = 4 * lane; w < kWords; w += 128)
          if (w < words) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 4 * w), "l"(f + w) : "memory");
      } else {
        for (int w = lane; w < kWords; w += 32)
          if (w < words) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4 * w), "l"(f + w) : "memory");
      }
    }
  }
  Group<int16_t, kW> count[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int v = v0 + (u * kThreads + tid) * kW;
#pragma unroll
    for (int k = 0; k < kW; ++k) count[u].x[k] = 0;
    if (P.counts && v < v1)
      count[u] = *reinterpret_cast<const Group<int16_t, kW>*>(P.counts + static_cast<size_t>(b) * P.V + v);
  }
  const int32_t* const from = warp == 0 ? P.tokens + static_cast<size_t>(b) * P.T : P.bias_tokens + static_cast<size_t>(b) * P.K;
  const int lists_most = warp == 0 ? (P.tokens && P.penalties ? P.T : 0) : (warp == 1 ? P.K : 0);
  const int next = lane < lists_most ? __ldg(from + lane) : -1;
  const float rep = P.rep ? __ldg(P.rep + b) : 1.0f, freq = P.freq ? __ldg(P.freq + b) : 0.0f;
  const float pres = P.pres ? __ldg(P.pres + b) : 0.0f;
  bool ok = true;
  if (P.parents && tid < P.N) {
    const int parent = __ldg(P.parents + static_cast<size_t>(b) * P.N + tid);
    up[tid] = parent;
    ok = tid >= m || (tid == 0 ? parent == -1 : (parent >= 0 && parent < tid));
  }
  for (int x = tid; x < kSpan / 32; x += kThreads) special[x] = 0;
  if (tid == 0) length = 0;
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!__syncthreads_and(ok && m >= 0 && m <= P.N) || first >= m) return;
  const int here = min(m - first, most);       // positions of this CTA
  // A chain's position i follows tokens 0 .. i - 1, a tree's node i follows its ancestors and itself.
  if (warp == 0) {
    const int have = gather(from, next, min(lists_most, P.parents ? m : m - 1), v0, v1, lane, said, said_at, special);
    if (lane == 0) lists[0] = have;
  } else if (warp == 1) {
    const int have = gather(from, next, lists_most, v0, v1, lane, biased, biased_at, special);
    if (lane == 0) lists[1] = have;
  } else if (P.parents && tid - 64 < m) {      // warps 2 to 4: places 1.. of the tree that a node follows, as bits from 0
    unsigned long long set = 0;
    for (int x = tid - 64; x > 0; x = up[x]) set |= 1ull << (x - 1);     // (parents lie below their nodes)
    above[tid - 64] = set;
  }

  T* const row = static_cast<T*>(P.logits) + (static_cast<size_t>(b) * P.N + first) * P.V + v0;
  if (P.mask) {
    const T barred = from_float<T>(__int_as_float(0xff800000));
    G all;
    Group<T, 4> all4;
    Group<T, 2> all2;
#pragma unroll
    for (int k = 0; k < kW; ++k) all.x[k] = barred;
#pragma unroll
    for (int k = 0; k < 4; ++k) all4.x[k] = all2.x[k & 1] = barred;
#pragma unroll 1
    for (int u = 0; u < kU; ++u) {
      const int at = (u * kThreads + tid) * kW;
      if (v0 + at >= v1) break;
      T* to = row + at;
#pragma unroll 2
      for (int y = 0; y < here; ++y, to += P.V) {
        unsigned bar = ~(masks[y][at >> 5] >> (at & 31)) & kAll;
        if (bar == kAll) {
          put(to, all);
        } else if (kW == 8 && bar) {
          // Barred in part. Where much is left of 16 or 32 bytes they are read and written whole (parts of them, without
          // reading: 66 us against 43 for 64 rows of 6 positions barred at random), else halves, quarters and single logits
          // are written (nearly all barred: 25 us against 28 with single logits).
          if (__popc(bar) > 2 && __popc(bar) < 7) {
            G z = *reinterpret_cast<const G*>(to);
#pragma unroll
            for (int k = 0; k < kW; ++k)
              if ((bar >> k) & 1) z.x[k] = barred;
            put(to, z);
            continue;
          }
#pragma unroll
          for (int h = 0; h < kW; h += 4) {
            if ((bar >> h & 15) == 15) {
              put(to + h, all4);
              continue;
            }
#pragma unroll
            for (int k = h; k < h + 4; k += 2) {
              const unsigned two = bar >> k & 3;
              if (two == 3) put(to + k, all2);
              else if (two) to[k + (two >> 1)] = barred;
            }
          }
        }
      }
    }
  }
  __syncthreads();

#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int at = (u * kThreads + tid) * kW;  // (behind the row's last token nothing is counted or special)
    const unsigned marks = special[at >> 5] >> (at & 31) & kAll;
    unsigned touched = marks;
#pragma unroll
    for (int k = 0; k < kW; ++k) touched |= (count[u].x[k] != 0 ? 1u : 0u) << k;
    if (!touched) continue;
    int to = atomicAdd(&length, __popc(touched));
#pragma unroll
    for (int k = 0; k < kW; ++k)
      if ((touched >> k) & 1) list[to++] = listed(at + k, (marks >> k) & 1, count[u].x[k]);
  }
  __syncthreads();

  // A token of the list a lane, at one position, or at more of them where the list is long: their logits are then in
  // flight together.
  const int len = length;
  if (len == 0) return;
  const int step = min(max(len * here / kThreads, 1), here), items = len * ((here + step - 1) / step);
  const unsigned inv = 0xffffffffu / len + 1;  // (x inv / 2^32 is x / len for x len < 2^32; 1 / 1 is 2^32)
  for (int x = tid; x < items; x += kThreads) {
    const int block = len == 1 ? x : __umulhi(x, inv), l = x - block * len;
    const int y0 = block * step, steps = min(step, here - y0);
    const unsigned e = list[l];
    const int place = e & (kSpecial - 1), n = (e >> 16) & 32767;
    T* const at = row + static_cast<size_t>(y0) * P.V + place;
    float z[kPositions];
    unsigned allowed = 0;                      // a bit a position
#pragma unroll
    for (int y = 0; y < kPositions; ++y) {
      if (y >= steps) break;
      if (P.mask && !((masks[y0 + y][place >> 5] >> (place & 31)) & 1)) continue;
      allowed |= 1u << y;
      z[y] = to_float<T>(at[static_cast<size_t>(y) * P.V]);
    }
    bool any = (e >> 16) != 0;                 // concerned at every position
    unsigned long long more = 0;               // what the round adds to n, seven bits a position
    float add = 0.0f;
    if (e & kSpecial) {
      for (int s = 0; s < lists[0]; ++s) {
        if (said[s] != place) continue;
        const int a = said_at[s];              // (place 0 of a tree, the root, is above every node)
        for (int y = 0; y < steps; ++y)
          if (P.parents ? a == 0 || ((above[first + y0 + y] >> (a - 1)) & 1) : a < first + y0 + y) more += 1ull << (7 * y);
      }
      for (int s = 0; s < lists[1]; ++s)
        if (biased[s] == place) {
          add += __ldg(P.bias + static_cast<size_t>(b) * P.K + biased_at[s]);
          any = true;
        }
    }
#pragma unroll
    for (int y = 0; y < kPositions; ++y) {
      if (y >= steps) break;
      const int uses = n + (static_cast<int>(more >> (7 * y)) & 127);
      if (!((allowed >> y) & 1) || !(any || uses > 0)) continue;
      float v = z[y];
      if (uses > 0 || e >> 31) v = v > 0.0f ? v / rep : v * rep;
      v -= freq * static_cast<float>(uses);
      if (uses > 0) v -= pres;
      at[static_cast<size_t>(y) * P.V] = from_float<T>(v + add);
    }
  }
}

template <typename T>
int launch_shape(ShapeParams& P, bool whole, int sms, cudaStream_t st) {
  // Blocks of at most kPositions positions, and so many that there are four CTAs an SM (8 rows of 5 positions, V 32000,
  // open masks: 9.2 us so, 12.3 with blocks of 5); two groups a thread where that still leaves eight (64 rows of 6 positions,
  // V 128256, narrow masks: 28 us so, 30 with one).
  const long long runs = static_cast<long long>(P.B) * ((P.V - 1) / (8 * kThreads) + 1);
  P.per = (P.N - 1) / ((P.N - 1) / kPositions + 1) + 1;
  if (runs * P.N < 4ll * sms * P.per) P.per = static_cast<int>(runs * P.N / (4ll * sms)) + 1;
  P.blocks = (P.N - 1) / P.per + 1;
  const bool two = whole && runs * P.blocks >= 16ll * sms;
  const int span = kThreads * (two ? 16 : 8);
  const long long grid = static_cast<long long>(P.B) * ((P.V + span - 1) / span) * P.blocks;
  if (grid > 0x7fffffffll) return SV_ERR_BAD_SHAPE;
  if (!whole) sv_shape_kernel<T, 1, 8><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(P);
  else if (two) sv_shape_kernel<T, 8, 2><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(P);
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
  P.mask = mask;
  P.mask_whole = words % 4 == 0 && !sv::misaligned(mask, 16);
  P.mask_row = static_cast<long long>(words) * mask_positions;
  P.mask_position = mask_positions == 1 ? 0 : static_cast<long long>(words);
  P.B = B;
  P.T = T;
  P.K = bias ? K : 0;
  P.N = N;
  P.V = V;
  if (!P.penalties && P.K == 0 && !mask) return SV_OK;
  const bool whole = V % 8 == 0 && !sv::misaligned(logits, 8 * size) && !sv::misaligned(P.counts, 16);
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  return dtype == SV_DTYPE_F32 ? launch_shape<float>(P, whole, sms, s) : launch_shape<__nv_bfloat16>(P, whole, sms, s);
}

extern "C" int spec_verify_count_tokens(const int32_t* tokens, const int32_t* num, int16_t* counts, int32_t prompt,
                                        int32_t B, int32_t M, int32_t V, void* cuda_stream) {
  if (!tokens || !counts) return SV_ERR_NULL_POINTER;
  if (B < 1 || B > (1 << 20) || M < 1 || M > (1 << 30) || V < 1 || V > (1 << 24)) return SV_ERR_BAD_SHAPE;
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
