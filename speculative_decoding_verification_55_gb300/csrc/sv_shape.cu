// Shaping of a round's logits before they are verified, and the token counts that it reads ([R] "Speculative
// decoding", rayaq.ca ml-models -- Why the output is exactly the target's: temperature, top-p and any penalties are
// applied to p and q before the test).
//
//   n = occurrences of token t in the row's output + among the round's tokens that position i follows,
//   z' = z / rep where z > 0, else z * rep, if n > 0 or t is in the prompt (else z);
//   z'' = z' - freq n - pres [n > 0], then t's biases added one by one in their order;  -inf where the mask bars t.
//
// In place, one launch. A CTA owns a run of a row's tokens at all of the round's positions, in two passes. First, 8
// neighbouring tokens a thread (16 bytes of counts, a byte of a mask, 16 or 32 bytes of logits): the tokens that
// penalties or biases concern go into a list, and what the masks bar is written, groups barred whole without being
// read. Then the list's tokens at each position, one a lane. (Worked on in the first pass, where a warp's 256 tokens
// hold one or two of them, they cost 269 us for 256 rows of 8 x 152064 fp32, bound by the instructions of idle lanes.)
// Bound: the writes of barred logits; else the reads of the counts and the sectors of the logits that change.
// Rounding: fp32 throughout, one rounding to the logits' type at the end. Logits that nothing changes keep their bits.

#include <cuda_bf16.h>

#include <algorithm>

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

// The round's tokens or the row's biases that fall into a CTA's tokens, in their order, with the biases' values; one warp.
__device__ __forceinline__ int gather(const int32_t* from, const float* values, int n, int v0, int v1, int lane,
                                      unsigned short* place, unsigned short* index, float* value, unsigned* special) {
  constexpr int kAtOnce = 4;
  int have = 0;
  for (int x0 = 0; x0 < n; x0 += 32 * kAtOnce) {
    int t[kAtOnce];
    float f[kAtOnce];
#pragma unroll
    for (int y = 0; y < kAtOnce; ++y) {
      const int x = x0 + 32 * y + lane;
      t[y] = x < n ? __ldg(from + x) : -1;
      f[y] = values && x < n ? __ldg(values + x) : 0.0f;
    }
#pragma unroll
    for (int y = 0; y < kAtOnce; ++y) {
      const bool in = t[y] >= v0 && t[y] < v1;         // (v0 >= 0: a token below 0 is in no CTA's)
      const unsigned all = __ballot_sync(sv::kFull, in);
      if (in) {
        const int at = have + __popc(all & ((1u << lane) - 1)), p = t[y] - v0;
        place[at] = static_cast<unsigned short>(p);
        index[at] = static_cast<unsigned short>(x0 + 32 * y + lane);
        if (values) value[at] = f[y];
        atomicOr(special + (p >> 5), 1u << (p & 31));
      }
      have += __popc(all);
    }
  }
  return have;
}

// A token of the list: its place in the CTA's run, and its count.
constexpr int kPlaceBits = 13;

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
  // The round's tokens and the biases in the run: places in it, in the round and among the biases; then, of the first of
  // each token, what it is (above the place's bits), its count, the places of the round that say it (a bit each, from place
  // 1 on); of all, the token's next bias (0: none).
  constexpr int kPlace = (1 << kPlaceBits) - 1, kFirst = 1, kRoot = 2, kBiased = 4;
  extern __shared__ float dyn[];               // (as many as the call has biases: what is not taken is left to the L1)
  const int listed = kMaxRound + P.K;
  float* const value = dyn;                    // [K]
  unsigned short* const places = reinterpret_cast<unsigned short*>(value + P.K);    // [listed]
  unsigned short* const indexes = places + listed;
  unsigned short* const biases = indexes + listed;
  int16_t* const counted = reinterpret_cast<int16_t*>(biases + listed);
  __shared__ unsigned long long match[kMaxRound];
  __shared__ int up[kMaxRound], lists[2], length;
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
    const int n = P.tokens && P.penalties ? (P.parents ? m : m - 1) : 0;
    const int have = gather(P.tokens + static_cast<size_t>(b) * P.T, nullptr, n, v0, v1, lane, places, indexes, nullptr, special);
    if (lane == 0) lists[0] = have;
  } else if (warp == 1) {
    const size_t at = static_cast<size_t>(b) * P.K;
    const int have = gather(P.bias_tokens + at, P.bias + at, P.K, v0, v1, lane, places + kMaxRound, indexes + kMaxRound, value, special);
    if (lane == 0) lists[1] = have;
  } else if (tid - 64 < m) {                   // warps 2 to 4: the places from 1 on that a position follows, as bits from 0
    const int i = tid - 64;
    unsigned long long set = P.parents || i == 0 ? 0 : (1ull << (i - 1)) - 1;
    if (P.parents)
      for (int x = i; x > 0; x = up[x]) set |= 1ull << (x - 1);          // (parents lie below their nodes)
    above[i] = set;
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

  const int ns = lists[0], nb = lists[1];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int at = (u * kThreads + tid) * kW;  // (behind the row's last token nothing is counted or special)
    unsigned touched = 0;
#pragma unroll
    for (int k = 0; k < kW; ++k) touched |= (count[u].x[k] != 0 ? 1u : 0u) << k;
    touched &= ~(special[at >> 5] >> (at & 31));
    if (!touched) continue;
    int to = atomicAdd(&length, __popc(touched));
#pragma unroll
    for (int k = 0; k < kW; ++k)
      if ((touched >> k) & 1) list[to++] = static_cast<unsigned>(at + k) | static_cast<unsigned>(static_cast<unsigned short>(count[u].x[k])) << 16;
  }
  // (Looked up by each token at each position, 316 rows of 6 positions with 276 biases and V 162 took 52 us; so 39.)
  for (int x = tid; x < ns + nb; x += kThreads) {
    const int e = x < ns ? x : kMaxRound + x - ns, place = places[e];
    int what = kFirst, next = 0;               // (its own bits above the place are not set yet, others' may be)
    unsigned long long bits = 0;
    for (int r = 0; r < ns; ++r) {
      if ((places[r] & kPlace) != place) continue;
      if (r < e) what = 0;
      const int a = indexes[r];
      if (a == 0) what |= kRoot;
      else bits |= 1ull << (a - 1);
    }
    for (int r = kMaxRound; r < e; ++r)
      if ((places[r] & kPlace) == place) what = 0;
    for (int r = kMaxRound + nb - 1; r > e && r >= kMaxRound; --r)   // (backwards and to its end: four reads at a time)
      if ((places[r] & kPlace) == place) next = r;
    if (what && (next > 0 || e >= kMaxRound)) what |= kBiased;
    places[e] = static_cast<unsigned short>(place | what << kPlaceBits);
    biases[e] = static_cast<unsigned short>(next);
    counted[e] = P.counts ? __ldg(P.counts + static_cast<size_t>(b) * P.V + v0 + place) : 0;
    if (e < kMaxRound) match[e] = bits;
  }
  __syncthreads();

  // A token of the list, or of the round's and the biases', a lane, at one position, or at more of them where there are
  // many: their logits are then in flight together.
  const int len = length, all = len + ns + nb;
  if (all == 0) return;
  const int step = min(max(all * here / kThreads, 1), here), items = all * ((here + step - 1) / step);
  const unsigned inv = 0xffffffffu / all + 1;  // (x inv / 2^32 is x / all for x all < 2^32; 1 / 1 is 2^32)
  for (int x = tid; x < items; x += kThreads) {
    const int block = all == 1 ? x : __umulhi(x, inv), l = x - block * all;
    const int y0 = block * step, steps = min(step, here - y0);
    int place, n, what = 0, bias = 0;          // bias: the token's first
    unsigned long long bits = 0;
    if (l < len) {
      place = list[l] & kPlace;
      n = static_cast<int>(list[l]) >> 16;
    } else {
      const int e = l - len < ns ? l - len : kMaxRound + l - len - ns;
      what = places[e] >> kPlaceBits;
      if (!(what & kFirst)) continue;
      place = places[e] & kPlace;
      n = counted[e];
      bias = e < kMaxRound ? biases[e] : e;
      if (e < kMaxRound) bits = match[e];
    }
    T* const at = row + static_cast<size_t>(y0) * P.V + place;
    float z[kPositions] = {};
    unsigned allowed = 0;                      // a bit a position
#pragma unroll
    for (int y = 0; y < kPositions; ++y) {
      if (y >= steps) break;
      if (P.mask && !((masks[y0 + y][place >> 5] >> (place & 31)) & 1)) continue;
      allowed |= 1u << y;
      z[y] = to_float<T>(at[static_cast<size_t>(y) * P.V]);
    }
    const bool prompt = n < 0;
    n &= 32767;
#pragma unroll
    for (int y = 0; y < kPositions; ++y) {
      if (y >= steps) break;
      if (!((allowed >> y) & 1)) continue;
      const int i = first + y0 + y;
      // (Place 0 of a tree, the root, is above every node; of a chain, before every position but its own.)
      int uses = n;
      if (what) uses += __popcll(bits & above[i]) + ((what & kRoot) && (P.parents || i > 0));
      if (!(uses > 0 || prompt || (what & kBiased))) {
        allowed &= ~(1u << y);
        continue;
      }
      float v = z[y];
      if (uses > 0 || prompt) v = v > 0.0f ? v / rep : v * rep;
      v -= freq * static_cast<float>(uses);
      if (uses > 0) v -= pres;
      z[y] = v;
    }
    for (; bias > 0; bias = biases[bias]) {    // (their sum, added once, would round and overflow in another way)
      const float f = value[bias - kMaxRound];
#pragma unroll
      for (int y = 0; y < kPositions; ++y) z[y] += f;
    }
#pragma unroll
    for (int y = 0; y < kPositions; ++y) {
      if (y >= steps) break;
      if ((allowed >> y) & 1) at[static_cast<size_t>(y) * P.V] = from_float<T>(z[y]);
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
  const unsigned g = static_cast<unsigned>(grid);
  const size_t bytes = static_cast<size_t>(P.K) * 4 + static_cast<size_t>(kMaxRound + P.K) * (4 * 2);
  if (!whole) sv_shape_kernel<T, 1, 8><<<g, kThreads, bytes, st>>>(P);
  else if (two) sv_shape_kernel<T, 8, 2><<<g, kThreads, bytes, st>>>(P);
  else sv_shape_kernel<T, 8, 1><<<g, kThreads, bytes, st>>>(P);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

// ------------------------------------------------------------------------------------------------
// Token counts
// ------------------------------------------------------------------------------------------------

constexpr int kPer = 4;                        // tokens of a thread at a time

// Adds n occurrences. The sum and its limit do not depend on the order in which threads come.
__device__ __forceinline__ void add_count(unsigned short* at, int n) {
  unsigned short old = __ldcg(at);
  for (;;) {                                   // ends: another thread's addition is what makes a turn fail
    const int sum = min((old & 32767) + n, 32767);
    const unsigned short now = atomicCAS(at, old, static_cast<unsigned short>((old & 0x8000) | sum));
    if (now == old) return;
    old = now;
  }
}

// Occurrences of a token among a warp's lanes are added once, by the first of them; kMany (long rows of output): into a
// table in shared memory, a slot's first token each, which goes to the counts at the end, other tokens at once. (Straight to
// the counts, 4 rows of 1,000,000 tokens took 12.8 ms, the warps with a frequent token retrying; so they take 0.6.)
constexpr int kSlots = 4096;
template <bool kPrompt, bool kMany>
__global__ void __launch_bounds__(kThreads) sv_count_kernel(const int32_t* tokens, const int32_t* num, int16_t* counts,
                                                            int M, int V, int chunks, int span) {
  __shared__ int held[kMany ? kSlots : 1], seen[kMany ? kSlots : 1];
  const int b = blockIdx.x / chunks, begin = (blockIdx.x - b * chunks) * span;
  const int m = num ? __ldg(num + b) : M;
  if (m > M || begin >= m) return;
  const int end = min(m, begin + span);
  unsigned short* const row = reinterpret_cast<unsigned short*>(counts) + static_cast<size_t>(b) * V;
  if (kMany) {
    for (int x = threadIdx.x; x < kSlots; x += kThreads) {
      held[x] = -1;
      seen[x] = 0;
    }
    __syncthreads();
  }
  for (int x0 = begin; x0 < end; x0 += kThreads * kPer) {
    int t[kPer];
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
      const int x = x0 + y * kThreads + threadIdx.x;
      t[y] = x < end ? __ldg(tokens + static_cast<size_t>(b) * M + x) : -1;
      if (static_cast<unsigned>(t[y]) >= static_cast<unsigned>(V)) t[y] = -1;
    }
    if constexpr (kPrompt) {
      unsigned short c[kPer];
#pragma unroll
      for (int y = 0; y < kPer; ++y) c[y] = t[y] >= 0 ? __ldcg(row + t[y]) : 0x8000;
#pragma unroll
      for (int y = 0; y < kPer; ++y)           // whoever writes a token in this call writes the same
        if (!(c[y] & 0x8000)) __stcg(row + t[y], static_cast<unsigned short>(c[y] | 0x8000));
    } else {
#pragma unroll
      for (int y = 0; y < kPer; ++y) {
        const unsigned same = __match_any_sync(sv::kFull, t[y]);
        if (t[y] < 0 || (threadIdx.x & 31) != __ffs(same) - 1) continue;
        const int n = __popc(same);
        if (kMany) {
          const int slot = t[y] % kSlots, was = atomicCAS(held + slot, -1, t[y]);
          if (was == -1 || was == t[y]) {
            atomicAdd(seen + slot, n);
            continue;
          }
        }
        add_count(row + t[y], n);
      }
    }
  }
  if constexpr (kMany) {
    __syncthreads();
    for (int x = threadIdx.x; x < kSlots; x += kThreads)
      if (seen[x]) add_count(row + held[x], seen[x]);
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
  // A CTA has as many tokens as leave eight CTAs an SM; its threads four at a time.
  constexpr int kBatch = kThreads * kPer;
  if (sv::misaligned(tokens, 4) || sv::misaligned(num, 4) || sv::misaligned(counts, 2)) return SV_ERR_MISALIGNED;
  const unsigned long long rows = B;
  if (sv::overlap({{counts, 2 * rows * V}}, {{tokens, 4 * rows * M}, {num, 4 * rows}})) return SV_ERR_OVERLAP;
  int dev = 0;
  const int st = sv::current_device_status(&dev);
  if (st != SV_OK) return st;
  const int sms = sv::device_sms(dev);
  if (sms < 1) return SV_ERR_CUDA;
  const long long batches = (M - 1) / kBatch + 1, turns = std::max(1ll, B * batches / (8ll * sms));
  const int span = static_cast<int>(std::min(turns, batches)) * kBatch;
  const int chunks = (M - 1) / span + 1;
  const long long grid = static_cast<long long>(B) * chunks;
  if (grid > 0x7fffffffll) return SV_ERR_BAD_SHAPE;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const unsigned g = static_cast<unsigned>(grid);
  if (prompt) sv_count_kernel<true, false><<<g, kThreads, 0, s>>>(tokens, num, counts, M, V, chunks, span);
  else if (batches > 1) sv_count_kernel<false, true><<<g, kThreads, 0, s>>>(tokens, num, counts, M, V, chunks, span);
  else sv_count_kernel<false, false><<<g, kThreads, 0, s>>>(tokens, num, counts, M, V, chunks, span);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
