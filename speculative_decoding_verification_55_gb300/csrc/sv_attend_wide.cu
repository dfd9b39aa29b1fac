// Attention of a round's tokens over the paged cache where a key head has more query rows than one
// 16-row matrix instruction holds (rounds and trees; the mathematics as in sv_attend.cu): the products
// run on the fifth-generation tensor cores with accumulators in tensor memory.
//
// One CTA per SM: a producer warp copying tiles of 128 entries from the pages, a warp whose one thread
// issues the matrix products, and two groups of four softmax warps. An item is up to 128 query rows of
// a key head; the groups take its tiles in turn, each with scores S [128 rows, 128 entries] and an
// accumulator O [128 rows, D] of its own in tensor memory (2 x (128 + D) of 512 columns), a thread per
// row. While one group computes the exponentials of its tile the tensor core multiplies the other's:
//   S = Q K^T        Q and K from shared memory;
//   P = 2^(c S - c m) in the cache's type, written over S, with the row's sum in fp32;
//   O += P V         P from tensor memory, V from shared memory.
// A row's m is its running maximum up to a slack of 2^8: the accumulator is only rescaled when the
// maximum has grown by more (probabilities up to 2^8 are as exact in both types, and the sums are
// fp32). The groups' parts are joined at the item's end, and the parts of several CTAs as in
// sv_attend.cu.
// Bound: the bytes of the cache. 128 x 128 x D products take about a third of the time that a tile's
// 4 x 128 x D bytes take from HBM, exponentials a sixth.

#include <cmath>

#include "sv_attend.cuh"

namespace {

using sv::AttendParams;
using sv::kFull;

constexpr int kTileLog2 = 7, kTile = 1 << kTileLog2;   // entries of a key tile
constexpr int kRows = 128;                             // query rows of an item
constexpr int kSoftWarps = 8, kSoft = 32 * kSoftWarps;
constexpr int kThreads = kSoft + 64;                   // and the producer's and the products' warps
constexpr int kProducer = kSoftWarps, kProducts = kSoftWarps + 1;
constexpr float kSlack = 8.0f;
constexpr int kColumns = 512;                          // tensor memory columns of the CTA

template <int D>
constexpr int kStageBytes = 2 * kTile * D * 2;
template <int D>
constexpr int kStageCount = D == 64 ? 6 : 3;
// The queries; after them the exchange of accumulators: 16 columns of 128 rows each way, then the
// rows' maxima and sums.
constexpr int kExchange = 2 * 16 * kRows * 4;
template <int D>
constexpr int kQueryBytes = kRows * D * 2 > kExchange + 2 * kRows * 8 ? kRows * D * 2 : kExchange + 2 * kRows * 8;
template <int D>
constexpr int kSmemBytes = 1024 + kStageCount<D> * kStageBytes<D> + kQueryBytes<D>;

__device__ __forceinline__ uint64_t matrix_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  // Start, leading and stride offsets in 16-byte units; version 1; 128-byte swizzle.
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(stride >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// fp32 accumulators, operands of one 16-bit type; M = 128; b_rows: B's rows are its contraction index.
template <bool F16>
__device__ __forceinline__ constexpr uint32_t product_desc(int n, bool b_rows) {
  return (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | (b_rows ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | ((kRows >> 4) << 24);
}

__device__ __forceinline__ void product_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(desc), "r"(add ? 1u : 0u) : "memory");
}
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(desc), "r"(add ? 1u : 0u) : "memory");
}
// The barrier gets an arrival when every product issued so far is done.
__device__ __forceinline__ void products_done(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define SV_R8(x, o) "=r"(x[o]), "=r"(x[o + 1]), "=r"(x[o + 2]), "=r"(x[o + 3]), "=r"(x[o + 4]), "=r"(x[o + 5]), "=r"(x[o + 6]), "=r"(x[o + 7])
#define SV_W8(x, o) "r"(x[o]), "r"(x[o + 1]), "r"(x[o + 2]), "r"(x[o + 3]), "r"(x[o + 4]), "r"(x[o + 5]), "r"(x[o + 6]), "r"(x[o + 7])
// 16, 32 or 64 columns of this thread's lane of tensor memory, loaded when the call returns (the wait
// is part of the statement, so that no use of the registers can move before it).
__device__ __forceinline__ void tm_load64(uint32_t* r, uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,"
      "%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : SV_R8(r, 0), SV_R8(r, 8), SV_R8(r, 16), SV_R8(r, 24), SV_R8(r, 32), SV_R8(r, 40), SV_R8(r, 48), SV_R8(r, 56)
      : "r"(at) : "memory");
}
__device__ __forceinline__ void tm_load32(uint32_t* r, uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : SV_R8(r, 0), SV_R8(r, 8), SV_R8(r, 16), SV_R8(r, 24) : "r"(at) : "memory");
}
__device__ __forceinline__ void tm_load16(uint32_t* r, uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : SV_R8(r, 0), SV_R8(r, 8) : "r"(at) : "memory");
}
__device__ __forceinline__ void tm_store32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(at), SV_W8(r, 0), SV_W8(r, 8), SV_W8(r, 16), SV_W8(r, 24) : "memory");
}
__device__ __forceinline__ void tm_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A bounded wait; the first that gives up makes every later one return at once.
__device__ __forceinline__ bool wait_unless_lost(uint32_t bar, uint32_t parity, volatile int* lost) {
  if (*lost) return false;
  if (sv::mbar_wait(bar, parity)) return true;
  *lost = 1;
  return false;
}

template <bool F16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    sv_attend_wide_kernel(const AttendParams P, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap) {
  constexpr int kStages = kStageCount<D>;
  constexpr int kScores = 0, kAccum = 2 * kTile;       // columns: S0, S1, O0, O1
  extern __shared__ unsigned char dyn[];
  __shared__ __align__(8) unsigned long long full[kStages], empty[kStages], s_full[2], p_ready[2], o_full, q_full, drained;
  __shared__ unsigned long long masks[sv::kMaxTreeNodes];
  __shared__ long long scan[kThreads / 32];
  __shared__ sv::Plan plan;
  __shared__ int bad_stage[kStages], sm_last, sm_flags, sm_lost;
  __shared__ uint32_t sm_tm;
  const sv::Round& R = P.R;
  const sv::Cache& C = R.C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = (sv::smem_addr(dyn) + 1023u) & ~1023u;
  const uint32_t qs = ring + kStages * kStageBytes<D>;
  unsigned char* const ring_p = dyn + (ring - sv::smem_addr(dyn));
  unsigned char* const qs_p = dyn + (qs - sv::smem_addr(dyn));
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      sv::mbar_init(sv::smem_addr(full + s), 1);
      sv::mbar_init(sv::smem_addr(empty + s), 1);
    }
    for (int w = 0; w < 2; ++w) {
      sv::mbar_init(sv::smem_addr(s_full + w), 1);
      sv::mbar_init(sv::smem_addr(p_ready + w), kSoftWarps / 2);
    }
    sv::mbar_init(sv::smem_addr(&o_full), 1);
    sv::mbar_init(sv::smem_addr(&drained), 1);
    sv::mbar_init(sv::smem_addr(&q_full), kSoftWarps);
    sm_lost = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kProducts) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(sv::smem_addr(&sm_tm)), "r"(static_cast<uint32_t>(kColumns)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    fence_before();
  }
  sv::make_plan<kThreads>(R, scan, &plan);
  sv::fill_unused(P, D, tid, kThreads);
  if (P.shared && tid == 0) P.shared[blockIdx.x].x = -1;
  fence_after();
  const uint32_t tm = sm_tm;
  volatile int* const lost = &sm_lost;

  sv::Walk W;
  W.begin(R, plan);
  if (warp == kProducer) {
    // ---- Copies: page numbers are read one tile ahead of the copies that need them.
    sv::TileLoader T;
    T.init(C, 2, kTileLog2);
    int issued = 0;
    while (!*lost && W.next(R)) {
      const int entries = W.w.n + W.w.m;
      int p = T.page(C, W.row, W.first, entries, lane);
      for (int t = W.first; t < W.first + W.count; ++t) {
        const int p_next = t + 1 < W.first + W.count ? T.page(C, W.row, t + 1, entries, lane) : -1;
        const int s = issued % kStages;
        const uint32_t bar = sv::smem_addr(full + s);
        if (issued >= kStages &&
            !__all_sync(kFull, wait_unless_lost(sv::smem_addr(empty + s), (issued / kStages - 1) & 1, lost)))
          break;
        const unsigned go = __ballot_sync(kFull, p >= 0), out = __ballot_sync(kFull, p == -2);
        if (lane == 0) {
          bad_stage[s] = out != 0;
          sv::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(go)) << (T.rows_log2 + 7));
        }
        __syncwarp();
        if (p >= 0) T.load(C, &kmap, &vmap, t, W.head, p, lane, ring + s * kStageBytes<D>, bar);
        ++issued;
        p = p_next;
      }
    }
    // No copy is in flight when the CTA ends.
    for (int x = issued < kStages ? 0 : issued - kStages; x < issued; ++x)
      sv::mbar_wait_drain(sv::smem_addr(full + x % kStages), (x / kStages) & 1);
  } else if (warp == kProducts) {
    // ---- Products, by one thread: scores run two tiles ahead of the products with the values.
    if (lane == 0) {
      constexpr uint32_t ds = product_desc<F16>(kTile, false), dp = product_desc<F16>(D, true);
      int base = 0, items = 0, ready[2] = {0, 0};
      auto scores = [&](int idx) {
        const int x = base + idx, s = x % kStages, w = idx & 1;
        if (!wait_unless_lost(sv::smem_addr(full + s), (x / kStages) & 1, lost)) return;
        fence_after();
        const uint32_t kb = ring + s * kStageBytes<D>;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          product_ss(tm + kScores + w * kTile,
                     matrix_desc(qs + (k >> 2) * (kRows * 128) + (k & 3) * 32, 16, 1024),
                     matrix_desc(kb + (k >> 2) * (kTile * 128) + (k & 3) * 32, 16, 1024), ds, k > 0);
        products_done(sv::smem_addr(s_full + w));
      };
      while (!*lost && W.next(R)) {
        if (!wait_unless_lost(sv::smem_addr(&q_full), items & 1, lost)) break;
        fence_after();
        scores(0);
        if (W.count > 1) scores(1);
        for (int idx = 0; idx < W.count && !*lost; ++idx) {
          const int x = base + idx, s = x % kStages, w = idx & 1;
          if (!wait_unless_lost(sv::smem_addr(p_ready + w), ready[w]++ & 1, lost)) break;
          fence_after();
          const uint32_t vb = ring + s * kStageBytes<D> + kTile * D * 2;
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            product_ts(tm + kAccum + w * D, tm + kScores + w * kTile + k * 8,
                       matrix_desc(vb + k * 2048, kTile * 128, 1024), dp, idx > 1 || k > 0);
          products_done(sv::smem_addr(empty + s));
          if (idx + 2 < W.count) scores(idx + 2);
        }
        products_done(sv::smem_addr(&o_full));
        base += W.count;
        ++items;
      }
      if (*lost) {              // products in flight end before the tensor memory is given back
        products_done(sv::smem_addr(&drained));
        sv::mbar_wait_drain(sv::smem_addr(&drained), 0);
      }
    }
    __syncwarp();
  } else {
    // ---- Softmax
    const int wg = warp >> 2, wq = warp & 3, row = 32 * wq + lane, wtid = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * wq) << 16;
    const uint32_t ts = tm + lanes + kScores + wg * kTile, to = tm + lanes + kAccum + wg * D;
    const float c = P.c;
    int base = 0, items = 0, seen_s = 0;
    while (W.next(R)) {
      const int n = W.w.n, m = W.w.m, entries = n + m;
      const int row0 = W.q_tile * kRows, rows = min(kRows, m * R.group - row0);
      const char* qb = P.q + W.row * P.row_stride + static_cast<long long>(W.head) * R.group * (D * 2);
      {
        constexpr int kEach = kRows * (D / 8) / kSoft;   // all of a thread's loads in flight at once
        uint4 v[kEach];
#pragma unroll
        for (int y = 0; y < kEach; ++y) {
          const int x = y * kSoft + tid, r = x / (D / 8), ch = x % (D / 8);
          v[y] = make_uint4(0u, 0u, 0u, 0u);
          if (r < rows) {
            const int i = (row0 + r) / R.group, hg = (row0 + r) - i * R.group;
            v[y] = __ldg(reinterpret_cast<const uint4*>(qb + i * P.token_stride + hg * (D * 2)) + ch);
          }
        }
#pragma unroll
        for (int y = 0; y < kEach; ++y) {
          const int x = y * kSoft + tid, r = x / (D / 8), ch = x % (D / 8);
          const uint32_t a = sv::swizzled(qs + (ch >> 3) * (kRows * 128), r, ch & 7);
          *reinterpret_cast<uint4*>(qs_p + (a - qs)) = v[y];
        }
      }
      if (tid == 0) sm_flags = 0;
      bool bad = false;
      const int last = W.first + W.count;
      const bool tail = last * kTile > n;      // the run reaches the round's own entries
      const int32_t* par = P.parents ? P.parents + static_cast<size_t>(W.row) * R.N : nullptr;
      if (par && tail) bad = !sv::tree_masks(par, m, masks, tid, kSoft);
      else if (par)
        for (int x = tid; x < m; x += kSoft) {
          const int p = __ldg(par + x);
          bad |= x == 0 ? p != -1 : (p < 0 || p >= x);
        }
      fence_async();
      fence_before();
      sv::named_bar_sync(1, kSoft);
      if (lane == 0) sv::mbar_arrive(sv::smem_addr(&q_full));
      const int tok = min((row0 + row) / R.group, m - 1);
      const bool active = 32 * wq < rows;      // the warp has a query row
      float mx = -INFINITY, l = 0.0f;
      bool odd = false;

      for (int idx = wg; idx < W.count; idx += 2) {
        const int x = base + idx, s = x % kStages;
        bool go = wait_unless_lost(sv::smem_addr(s_full + wg), seen_s++ & 1, lost);
        go = go && wait_unless_lost(sv::smem_addr(full + s), (x / kStages) & 1, lost);
        if (!__all_sync(kFull, go)) break;
        fence_after();
        bad |= bad_stage[s] != 0;
        const int j0 = (W.first + idx) * kTile;
        const bool edge = j0 + kTile > n;      // entries of the round itself, or behind the last
        if (active) {
          // 64 scores at a time, read twice: for the maximum, then for the exponentials (all 128 at
          // once would not fit the registers).
          const uint64_t see[2] = {edge ? sv::seen_bits(j0 - n, tok, par ? masks[tok] : ~0ull, par) : ~0ull,
                                   edge ? sv::seen_bits(j0 + 64 - n, tok, par ? masks[tok] : ~0ull, par) : ~0ull};
          auto load = [&](uint32_t (&sc)[64], int y) {
            tm_load64(sc, ts + y);
            if (!edge) return;
            const uint32_t lo = static_cast<uint32_t>(see[y >> 6]), hi = static_cast<uint32_t>(see[y >> 6] >> 32);
#pragma unroll
            for (int z = 0; z < 32; ++z) {
              if (!((lo >> z) & 1)) sc[z] = 0xff800000u;
              if (!((hi >> z) & 1)) sc[32 + z] = 0xff800000u;
            }
          };
          float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int y = 0; y < kTile; y += 64) {
            uint32_t sc[64];
            load(sc, y);
#pragma unroll
            for (int z = 0; z < 64; ++z) v[z & 3] = fmaxf(v[z & 3], __uint_as_float(sc[z]));
          }
          const float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
          // The first tile sets the maximum; later ones move it when it has grown by over kSlack.
          const bool grew = top > mx && (mx == -INFINITY || (top - mx) * c > kSlack);
          if (__any_sync(kFull, grew)) {
            const float f = !grew ? 1.0f : (mx == -INFINITY ? 0.0f : sv::ex2((mx - top) * c));
            if (grew) mx = top;
            l *= f;
            if (idx > 1) {                     // products with earlier tiles' values are done
#pragma unroll
              for (int y = 0; y < D; y += 32) {
                uint32_t o[32];
                tm_load32(o, to + y);
#pragma unroll
                for (int z = 0; z < 32; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * f);
                tm_store32(to + y, o);
              }
            }
          }
          const float b = mx == -INFINITY ? 0.0f : -mx * c;
          const sv::f32x2 c2 = sv::pk(c, c), b2 = sv::pk(b, b);
          sv::f32x2 sum[2] = {sv::pk(0.0f, 0.0f), sv::pk(0.0f, 0.0f)};
#pragma unroll
          for (int y = 0; y < kTile; y += 64) {
            uint32_t sc[64], p[32];
            load(sc, y);
#pragma unroll
            for (int z = 0; z < 32; ++z) {
              float p0, p1;
              sv::upk(sv::fma2(sv::pk(__uint_as_float(sc[2 * z]), __uint_as_float(sc[2 * z + 1])), c2, b2), p0, p1);
              p0 = sv::ex2(p0);
              p1 = sv::ex2(p1);
              sum[z & 1] = sv::add2(sum[z & 1], sv::pk(p0, p1));
              p[z] = sv::pack2<F16>(p0, p1);
            }
            tm_store32(ts + y / 2, p);
          }
          float s0, s1;
          sv::upk(sv::add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
          tm_wait_store();
        }
        if (edge) {
          // Value rows of the round's own entries: what is not finite is cleared; rows behind the last
          // entry are cleared whole.
          unsigned char* vb = ring_p + s * kStageBytes<D> + kTile * D * 2;
          const int r0 = max(n - j0, 0);
          for (int y = r0 * (D / 8) + wtid; y < kTile * (D / 8); y += 128) {
            const int r = y / (D / 8), ch = y % (D / 8);
            uint4* at = reinterpret_cast<uint4*>(vb + (ch >> 3) * (kTile * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            bool clear = true;
            if (j0 + r < entries) {
              clear = false;
              v = *at;
              v.x = sv::finite2<F16>(v.x, ~0u, clear);
              v.y = sv::finite2<F16>(v.y, ~0u, clear);
              v.z = sv::finite2<F16>(v.z, ~0u, clear);
              v.w = sv::finite2<F16>(v.w, ~0u, clear);
              odd |= clear;
            }
            if (clear) *at = v;
          }
        }
        if (edge) fence_async();
        fence_before();
        __syncwarp();
        if (lane == 0) sv::mbar_arrive(sv::smem_addr(p_ready + wg));
      }
      wait_unless_lost(sv::smem_addr(&o_full), items & 1, lost);
      fence_after();
      if (bad || *lost) atomicOr(&sm_flags, 1);
      if (odd) atomicOr(&sm_flags, 2);
      base += W.count;
      ++items;

      // The two groups' parts of a row: each group finishes half of the columns.
      float2* ml = reinterpret_cast<float2*>(qs_p + kExchange);       // [2][kRows]
      float* give = reinterpret_cast<float*>(qs_p) + wg * 16 * kRows; // [16][kRows]
      const float* take = reinterpret_cast<const float*>(qs_p) + (wg ^ 1) * 16 * kRows;
      sv::named_bar_sync(1, kSoft);            // the queries have been read
      ml[wg * kRows + row] = make_float2(mx, l);
      const int flags = sm_flags;
      sv::named_bar_sync(1, kSoft);
      const float2 other = ml[(wg ^ 1) * kRows + row];
      const float jm = fmaxf(mx, other.x);
      const float mine = mx == -INFINITY ? 0.0f : sv::ex2((mx - jm) * c);
      float jl = (mx == -INFINITY ? l : l * mine) +
                 (other.x == -INFINITY ? other.y : other.y * sv::ex2((other.x - jm) * c));
      if (flags & 1) jl = __int_as_float(0x7fffffff);
      const bool any = W.count > wg;           // the group had a tile: its accumulator is set
      const bool whole = W.count == W.w.tiles;
      const int slot = 2 * blockIdx.x + (W.first == 0 ? 1 : 0);
      const int i = (row0 + row) / R.group, hq = W.head * R.group + (row0 + row) - i * R.group;
      const size_t at = (static_cast<size_t>(W.row) * R.N + i) * P.Hq + hq;
      const float inv = 1.0f / jl;
      for (int k = 0; k < D / 32; ++k) {
        const int mycol = wg * (D / 2) + 16 * k, theirs = (wg ^ 1) * (D / 2) + 16 * k;
        uint32_t g[16], o[16];
        tm_load16(g, to + theirs);
        tm_load16(o, to + mycol);
#pragma unroll
        for (int z = 0; z < 16; ++z) give[z * kRows + row] = any ? __uint_as_float(g[z]) * mine : 0.0f;
        sv::named_bar_sync(1, kSoft);
        float f[16];
#pragma unroll
        for (int z = 0; z < 16; ++z)
          f[z] = (any ? __uint_as_float(o[z]) * mine : 0.0f) + take[z * kRows + row];
        // Values that are not finite were left out of the products, where a zero probability would have
        // made NaN of them: they are added to the rows that attend them.
        if (flags & 2) {
          for (int j = max(n, W.first * kTile); j < min(entries, last * kTile); ++j) {
            const int page = sv::cache_page(C, W.row, j), a = j - n;
            if (!sv::page_ok(C, page)) continue;
            if (!(par ? a <= 0 || ((masks[tok] >> (a - 1)) & 1) : a <= tok)) continue;
            const unsigned short* v = reinterpret_cast<const unsigned short*>(C.v + sv::entry_offset(C, page, W.head, j)) + mycol;
#pragma unroll
            for (int z = 0; z < 16; ++z) {
              const float e = sv::value_of<F16>(v[z]);
              if (!isfinite(e)) f[z] += e;
            }
          }
        }
        if (row < rows) {
          if (whole) {
            uint32_t p[8];
#pragma unroll
            for (int z = 0; z < 8; ++z) p[z] = sv::pack2<F16>(f[2 * z] * inv, f[2 * z + 1] * inv);
            uint4* out = reinterpret_cast<uint4*>(static_cast<char*>(P.out) + (at * D + mycol) * 2);
            out[0] = make_uint4(p[0], p[1], p[2], p[3]);
            out[1] = make_uint4(p[4], p[5], p[6], p[7]);
          } else {
            float4* out = reinterpret_cast<float4*>(P.part_o + (static_cast<size_t>(slot) * kRows + row) * D + mycol);
#pragma unroll
            for (int z = 0; z < 4; ++z) out[z] = make_float4(f[4 * z], f[4 * z + 1], f[4 * z + 2], f[4 * z + 3]);
          }
        }
        sv::named_bar_sync(1, kSoft);
      }
      if (wg == 0 && row < rows) {
        if (!whole) P.part_ml[slot * kRows + row] = make_float2(jm, jl);
        else if (P.lse) P.lse[at] = (jm * c + log2f(jl)) * 0.6931471805599453f;
      }
      if (whole) continue;
      sv::join_parts<F16, D, kRows, kSoft>(P, W, plan, row0, rows, tid, reinterpret_cast<float*>(qs_p), &sm_last);
    }
    fence_before();
  }
  __syncthreads();
  if (warp == kProducts) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                 ::"r"(tm), "r"(static_cast<uint32_t>(kColumns)) : "memory");
  }
}

template <bool F16, int D>
int launch(const AttendParams& P, const CUtensorMap& k, const CUtensorMap& v, int grid, cudaStream_t st) {
  auto kern = sv_attend_wide_kernel<F16, D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<D>) != cudaSuccess)
    return SV_ERR_CUDA;
  kern<<<grid, kThreads, kSmemBytes<D>, st>>>(P, k, v);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace

namespace sv {

int launch_attend_wide(const AttendParams& P, bool f16, const CUtensorMap& k, const CUtensorMap& v, int grid,
                       cudaStream_t st) {
  if (P.R.C.head_dim == 64) return f16 ? launch<true, 64>(P, k, v, grid, st) : launch<false, 64>(P, k, v, grid, st);
  return f16 ? launch<true, 128>(P, k, v, grid, st) : launch<false, 128>(P, k, v, grid, st);
}

}  // namespace sv
