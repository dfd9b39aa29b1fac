// Attention of a round's tokens over the paged cache where a key head has more query rows than one
// 16-row matrix instruction holds (rounds and trees; the mathematics as in sv_attend.cu): the products
// run on the fifth-generation tensor cores with accumulators in tensor memory.
//
// One CTA per SM: two warps copying tiles of 128 entries from the pages, a warp whose one thread
// issues the matrix products, a warp that copies an item's queries and tells the others what the item is,
// and eight softmax warps. An item is up to 128 query rows of a key head, or two such query tiles at once. (A warp
// takes 48 ns to issue a box: one alone took 1.55 us for a tile from pages of 16, in boxes of 2 KB, longer than the
// tile takes from HBM.)
// Tensor memory holds the scores S [128 rows, 128 entries] of two tiles, or of one for each of two query tiles, and
// an accumulator O [128 rows, D] a query tile: 2 x 128 + D or 2 x 128 + 2 D of 512 columns (key tiles of heads of 256
// have 64 entries: 2 x 64 + 256).
//   S = Q K^T        Q and K from shared memory, up to two tiles ahead;
//   P = 2^(c S - c m) in the cache's type, written over S, with the row's sum in fp32;
//   O += P V         P from tensor memory, V from shared memory.
// Two threads share a row, 64 entries each, and meet once a tile for its maximum (two query tiles: a thread has a
// row). A row's m is its running maximum up to a slack of 2^8: the accumulator is only rescaled when the maximum has
// grown by more, a published method (probabilities above 1 are as exact, and the sums are fp32). The parts of several
// CTAs are joined as in sv_attend.cu.
// Bound: the bytes of the cache. The 128 x 128 x D products of a tile take about a third of the time
// that its 4 x 128 x D bytes take from HBM. With two groups of warps on a tile each (a row a thread, two
// accumulators, S and P sharing one buffer a group) a tile's chain of S, softmax, P V and the next S took
// 3900 cycles, two tiles at a time; here 128 rows take 1700 to 2000. Keys and values have slots of the ring
// of their own, given back when their product is done: with one slot for both, the products waited for
// the next keys before they gave back the last values (19 rows of 8000 entries: 172 us against 118).

#pragma once

#include <cmath>

#include "sv_attend.cuh"
#include "sv_tmem.cuh"

namespace {

using sv::ParamsOf;
using namespace sv::tmem;
using sv::kFull;

constexpr int kRows = 128;                             // query rows of a product
constexpr int kSoftWarps = 8, kSoft = 32 * kSoftWarps;
constexpr int kCopyWarps = 2;
constexpr int kThreads = kSoft + 32 * (kCopyWarps + 2);   // and the copies', the products' and the items' warps
constexpr int kCopies = kSoftWarps, kItems = kCopies + kCopyWarps, kProducts = kItems + 1;
constexpr int kScores = 2;                             // buffers of scores in tensor memory
constexpr int kPieces = 8;                             // items that the warps may be apart, and one

// kWays: query tiles of 128 rows that a CTA works on at once.
template <int D, int kWays>
struct Shape {
  static constexpr int kTileLog2 = D == 256 ? 6 : 7, kTile = 1 << kTileLog2;   // entries of a key tile
  static constexpr int kSlotBytes = kTile * D * 2;     // a tile's keys or its values
  static constexpr int kQueryBytes = kWays * kRows * D * 2;
  static constexpr int kSlots = D == 64 ? 12 : (D == 128 && kWays == 1 ? 6 : 5);   // keys and values in turn
  static constexpr int kAccum = kScores * kTile;       // tensor memory columns: S0, S1, then an O a way
  static constexpr int kChunk = D == 256 ? 32 : 64;    // scores of a thread in registers
  static_assert(kAccum + kWays * D <= kColumns, "tensor memory");
};

// An item, or a CTA's part of one, as the items' warp found it: read from shared memory by the others, so
// that none of them waits for lengths from global memory (2 us a load while the cache streams).
struct Item {
  int row, head, q_tile, first, count;                 // count 0: the end
  int n, m, tiles;
  int tokens, token0;                                  // the query tokens, and the first of them among the batch's
  long long item_at;
};

// Shared memory behind the ring and the queries.
template <int kSlots>
struct Control {
  unsigned long long full[kSlots], empty[kSlots], s_full[kScores], p_ready[kScores], o_full, q_full,
      q_empty, told[kPieces], drained;
  long long scan[kThreads / 32];
  sv::Plan plan;
  Item items[kPieces];
  float row_max[2][2][kRows];                          // by the tile's parity and half
  int bad[kCopyWarps][kPieces], armed[kCopyWarps], flags, lost;
  uint32_t tm;
};
template <int D, int kWays>
constexpr int kSmemBytes = Shape<D, kWays>::kSlots * Shape<D, kWays>::kSlotBytes + Shape<D, kWays>::kQueryBytes +
                           sizeof(Control<Shape<D, kWays>::kSlots>);

// For the merge kernel: what there is to the rows.
__device__ __forceinline__ void tell_rows(const sv::SharedParams& P, int tid) {
#pragma unroll 1
  for (int b = tid * gridDim.x + blockIdx.x; b < P.R.B; b += 32 * kCopyWarps * gridDim.x) P.rows[b] = sv::row_of_group(P.R, b);
}

// 32 bytes at once: a thread's own row, whose neighbours are other threads'.
__device__ __forceinline__ void store8(float* at, const float* f) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               ::"l"(at), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]) : "memory");
}

// kShared: a batch whose rows share the fronts of their contexts (SharedRound); an item's result, whole or a part, then
// goes to the merge kernel. Where two ways are for the fronts' many queries, an item of one query tile (a row's own
// entries) is worked on as with one way: two threads a row, two tiles ahead. (With its tiles in turn on both ways, each
// with a maximum, a sum and an accumulator of its own, 512 such items of 4 or 5 tiles took 42 us of the batch's 76.)
template <bool F16, int D, int kWays, bool kShared>
__global__ void __launch_bounds__(kThreads, 1)
    sv_attend_wide_kernel(const ParamsOf<kShared> P, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap,
                          const __grid_constant__ CUtensorMap qmap, int q_tokens) {
  using H = Shape<D, kWays>;
  constexpr int kSlots = H::kSlots, kTile = H::kTile, kAccum = H::kAccum;
  constexpr float kBits = sv::kProbBits<F16, true>;
  constexpr bool kOne = kShared && kWays == 2;         // items of one way among those of two
  extern __shared__ __align__(1024) unsigned char dyn[];
  auto& S = *reinterpret_cast<Control<kSlots>*>(dyn + kSlots * H::kSlotBytes + H::kQueryBytes);
  const auto& R = P.R;
  const sv::Cache& C = R.C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = sv::smem_addr(dyn), qs = ring + kSlots * H::kSlotBytes;
  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      sv::mbar_init(sv::smem_addr(S.full + s), kCopyWarps);
      sv::mbar_init(sv::smem_addr(S.empty + s), 1);
    }
    for (int w = 0; w < kScores; ++w) {
      sv::mbar_init(sv::smem_addr(S.s_full + w), 1);
      sv::mbar_init(sv::smem_addr(S.p_ready + w), kOne ? kSoftWarps : kSoftWarps / kWays);
    }
    sv::mbar_init(sv::smem_addr(&S.o_full), 1);
    sv::mbar_init(sv::smem_addr(&S.drained), 1);
    sv::mbar_init(sv::smem_addr(&S.q_full), 1);
    sv::mbar_init(sv::smem_addr(&S.q_empty), 1);
    for (int x = 0; x < kPieces; ++x) sv::mbar_init(sv::smem_addr(S.told + x), 1);
    S.lost = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kProducts) tm_alloc(&S.tm);
  if constexpr (kShared) asm volatile("griddepcontrol.wait;" ::: "memory");   // the packed tokens
  sv::make_plan<kThreads>(R, S.scan, &S.plan);
  asm volatile("griddepcontrol.launch_dependents;");   // the join kernel's CTAs, which wait for this grid's end
  if (!kShared && tid < kWays && !P.by_item) P.shared[blockIdx.x * kWays + tid].x = -1;
  fence_after();
  const uint32_t tm = S.tm;
  volatile int* const lost = &S.lost;

  // Whether an item is worked on with one way: always, never, or where it has one query tile.
  auto one_way = [&](const Item& I) {
    return kWays == 1 || (kOne && I.tokens * R.group - I.q_tile * kWays * P.tile_rows <= P.tile_rows);
  };
  // The next item's description. The items' warp always tells an end, however its own waits end: this wait is longer than
  // they can be, so that all warps know of the same items and meet at the same barriers.
  auto told = [&](int k) {
    Item I;
    if (sv::mbar_wait_drain(sv::smem_addr(S.told + k % kPieces), (k / kPieces) & 1)) I = S.items[k % kPieces];
    else {
      I.count = 0;
      *lost = 1;
    }
    return I;
  };
  if (warp >= kCopies && warp <= kItems) {
    // ---- Items, and their copies. These warps walk the items by the same instructions: a kernel's first pass
    // through any code waits for it to come from memory, and a walk of each warp's own took 2 us more.
    sv::WalkOf<kShared> W;
    W.begin(R, S.plan);
    sv::TileLoader T;
    T.init(C, 1, H::kTileLog2);
    const int mine = warp - kCopies, op = kCopyWarps * lane + mine;   // the boxes are divided among the copy warps
    int armed = 0, items = 0;                  // slots (tile x: 2 x and 2 x + 1) and items so far
    bool gone = false;
    for (;; ++items) {
      const bool more = !gone && W.next(R);
      if (warp == kItems) {
        // The item's description, then, the score products of the one before being done, its queries:
        // q_tokens tokens of the key head's query heads as rows.
        if (lane == 0) {
          int token0 = W.row * R.N;
          if constexpr (kShared) token0 = W.w.token0;
          S.items[items % kPieces] = Item{W.row, W.head, W.q_tile, W.first, more ? W.count : 0, W.w.n, W.w.m,
                                          W.w.tiles, sv::tokens_of(W.w), token0, W.item_at};
          sv::mbar_arrive(sv::smem_addr(S.told + items % kPieces));
        }
        if (!more) break;
        if (items > 0 &&
            !__all_sync(kFull, wait_unless_lost(sv::smem_addr(&S.q_empty), (items - 1) & 1, lost))) {
          gone = true;                         // the next turn tells the end
          continue;
        }
        if (lane == 0) {
          sv::mbar_arrive_expect_tx(sv::smem_addr(&S.q_full), kWays * q_tokens * R.group * D * 2);
          int token = 0, row = W.row;          // (of rows that share fronts, q is one row of all tokens)
          if constexpr (kShared) {
            token = W.w.token0;
            row = 0;
          }
          for (int x = 0; x < kWays * (D / 64); ++x)
            sv::tma_load(qs + x * (kRows * 128), &qmap, x % (D / 64) * 64, W.head * R.group,
                         token + (W.q_tile * kWays + x / (D / 64)) * (P.tile_rows / R.group), row, sv::smem_addr(&S.q_full));
        }
        ++armed;
        continue;
      }
      if (!more) break;
      const int entries = W.w.n + W.w.m;
      const int last = W.first + W.count;
      const int32_t* const table = sv::pages_of(R, W.row, W.w);
      sv::PagesAhead pages;
      pages.begin(T, C, table, W.first, last, entries, op);
      if (lane == 0) S.bad[mine][items % kPieces] = 0;
      for (int t = W.first; t < last && !gone; ++t) {
        const int p = pages.next(T, C, table, t, last, entries, op);
        const unsigned go = __ballot_sync(kFull, p >= 0), out = __ballot_sync(kFull, p == -2);
        if (lane == 0 && out) S.bad[mine][items % kPieces] = 1;
#pragma unroll
        for (int array = 0; array < 2; ++array) {
          const int e = armed, s = e % kSlots;
          const uint32_t bar = sv::smem_addr(S.full + s);
          if (e >= kSlots &&
              !__all_sync(kFull, wait_unless_lost(sv::smem_addr(S.empty + s), (e / kSlots - 1) & 1, lost))) {
            gone = true;
            break;
          }
          if (lane == 0) sv::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(go)) << (T.rows_log2 + 7));
          __syncwarp();
          if (p >= 0) T.load(C, array ? &vmap : &kmap, nullptr, t, W.head, p, op, ring + s * H::kSlotBytes, bar);
          ++armed;
        }
      }
    }
    // No copy is in flight when the CTA ends.
    if (warp == kItems) {
      if (armed > 0) sv::mbar_wait_drain(sv::smem_addr(&S.q_full), (armed - 1) & 1);
    } else {
      if constexpr (kShared) tell_rows(P, op);  // while the last tiles are computed
      else sv::fill_unused(P, D, op, 32 * kCopyWarps);
      // A slot is full when both warps have armed it. One whose wait gave up may be behind the other (by at most the
      // ring: the other's slots were given back full): it arrives for the slots that it has not armed.
      if (lane == 0) S.armed[mine] = armed;
      __syncwarp();
      sv::named_bar_sync(6, 32 * kCopyWarps);
      const int most = max(S.armed[0], S.armed[1]);
      if (lane == 0)
        for (int e = armed; e < most; ++e) sv::mbar_arrive(sv::smem_addr(S.full + e % kSlots));
      for (int e = max(0, most - kSlots); e < most; ++e)
        sv::mbar_wait_drain(sv::smem_addr(S.full + e % kSlots), (e / kSlots) & 1);
    }
  } else if (warp == kProducts) {
    // ---- Products, by one thread. Score buffer w of tile x: one way, w = x % 2, two tiles ahead of the
    // products with the values; two ways, w the way, a tile ahead.
    if (lane == 0) {
      // This thread's own instructions take much of a tile's time (100 cycles a wait, 60 a product): places in
      // the ring and barriers are counted on, not computed.
      constexpr uint32_t ds = product_desc<F16>(kTile, false), dp = product_desc<F16>(D, true);
      const uint32_t full = sv::smem_addr(S.full), empty = sv::smem_addr(S.empty);
      const uint32_t s_full = sv::smem_addr(S.s_full), p_ready = sv::smem_addr(S.p_ready);
      const Matrix ring_k = matrix(ring, 16, 1024), ring_v = matrix(ring, kTile * 128, 1024), queries = matrix(qs, 16, 1024);
      struct Place {
        int slot;
        uint32_t phase;
        __device__ __forceinline__ void step() {         // to the same array of the next tile
          slot += 2;
          if (slot >= kSlots) {
            slot -= kSlots;
            phase ^= 1u;
          }
        }
      } pk{0, 0u}, pv{1, 0u};
      uint32_t ws = 0, wp = 0, turn = 0;                 // score buffers next written and next read, and its phase (a bit a way)
      int items = 0, left = 0;                           // left: score products of the item still to come
      bool one = kWays == 1;                             // the item has one way
      auto scores = [&](int way) {                       // (one way of two: the score buffer)
        if ((way == 0 || one) && !wait_unless_lost(full + 8 * pk.slot, pk.phase, lost)) return;
        fence_after();
        const uint32_t w = kWays == 2 ? way : ws;
        const Matrix km = ring_k.at(pk.slot * H::kSlotBytes), qm = queries.at(one ? 0 : way * (kRows * D * 2));
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          product_ss(tm + w * kTile, qm.at((k >> 2) * (kRows * 128) + (k & 3) * 32),
                     km.at((k >> 2) * (kTile * 128) + (k & 3) * 32), ds, k > 0);
        products_done(s_full + 8 * w);
        if (way + 1 < kWays && !one) return;
        products_done(empty + 8 * pk.slot);
        pk.step();
        ws ^= 1;
        if (--left == 0) products_done(sv::smem_addr(&S.q_empty));
      };
      constexpr int kAhead = kWays == 2 ? 1 : kScores;
      for (;;) {
        const Item I = told(items);
        const int count = I.count;
        one = one_way(I);
        if (count == 0 || !wait_unless_lost(sv::smem_addr(&S.q_full), items & 1, lost)) break;
        left = count;
        for (int idx = -kAhead; idx < count; ++idx) {      // (below 0: the first score products alone)
          if (idx >= 0 && !wait_unless_lost(full + 8 * pv.slot, pv.phase, lost)) break;
          const Matrix vm = ring_v.at(pv.slot * H::kSlotBytes);
#pragma unroll 1
          for (int way = 0; way < kWays; ++way) {
            if (idx >= 0) {
              if (kWays == 2 && one && way != (idx & 1)) continue;
              const uint32_t w = kWays == 2 ? way : wp;
              if (!wait_unless_lost(p_ready + 8 * w, kWays == 2 ? turn >> way & 1 : turn, lost)) break;
              fence_after();
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k)
                product_ts(tm + kAccum + (one ? 0 : way * D), tm + w * kTile + k * 8, vm.at(k * 2048), dp, idx > 0 || k > 0);
              if (way + 1 == kWays || one) products_done(empty + 8 * pv.slot);
              if (kWays == 2) turn ^= 1u << way;
            }
            if (left > 0) scores(way);
          }
          if (idx < 0) continue;
          pv.step();
          wp ^= 1;
          if (kWays == 1 && wp == 0) turn ^= 1u;
        }
        if (*lost) break;
        products_done(sv::smem_addr(&S.o_full));
        ++items;
      }
    }
    __syncwarp();
  } else {
    // ---- Softmax
    const int wq = warp & 3, row = 32 * wq + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * wq) << 16;
    const float c = P.c;
    int base = 0, items = 0;                   // tiles before the item
    int used[2] = {0, 0};                      // uses of the score buffers (two ways)
    for (;;) {
      const Item W = told(items);
      if (W.count == 0) break;
      // One way: two warps share rows, `half` a tile's entries and D each. Two ways: four warps have a way.
      const bool one = one_way(W);
      const int half = one ? warp >> 2 : 0, way = one ? 0 : warp >> 2;
      const int cols = one ? kTile / 2 : kTile, outs = one ? D / 2 : D;     // scores and columns of O of a thread
      const uint32_t to = tm + lanes + kAccum + way * D + half * outs;
      const int n = W.n, m = W.m, entries = n + m;
      const int row0 = (W.q_tile * kWays + way) * P.tile_rows, rows = min(P.tile_rows, W.tokens * R.group - row0);
      if (tid == 0) S.flags = 0;                // nobody sets one before this thread's first tile is used
      const int last = W.first + W.count;
      int side = 0;
      const int32_t* par = nullptr;
      if constexpr (kShared) {
        side = W.row >= R.groups;
        if (P.parents && side) par = P.parents + static_cast<size_t>(W.row - R.groups) * R.N;
      } else if (P.parents) {
        par = P.parents + static_cast<size_t>(W.row) * R.N;
      }
      bool bad = false;                        // the row's tree is not valid (a thread a node), or a page
      if (par && tid < m) {
        const int p = __ldg(par + tid);
        bad = tid == 0 ? p != -1 : (p < 0 || p >= tid);
      }
      const int tok = min((row0 + row) / R.group, m - 1);
      const bool active = 32 * wq < rows;      // the warp has a query row
      const unsigned long long mask = par && last * kTile > n ? sv::tree_mask(par, tok) : 0ull;
      float mx = -INFINITY, l = 0.0f;
      bool odd = false;

      for (int idx = 0; idx < W.count; ++idx) {
        const int x = base + idx, s = (2 * x + 1) % kSlots;
        const int w = kWays == 1 ? x % kScores : (one ? idx & 1 : way);
        const int turn = kWays == 1 ? x / kScores : (w ? used[1]++ : used[0]++);
        const int j0 = (W.first + idx) * kTile;
        const bool edge = j0 + kTile > n;      // entries of the round itself, or behind the last
        bool go = wait_unless_lost(sv::smem_addr(S.s_full + w), turn & 1, lost);
        if (edge || idx + 1 == W.count)        // the values are in, and the producer has seen all pages
          go = go && wait_unless_lost(sv::smem_addr(S.full + s), ((2 * x + 1) / kSlots) & 1, lost);
        if (!__all_sync(kFull, go)) {          // a wait gave up: the barriers alone
          if (active && one) sv::named_bar_sync(2 + wq, 64);
          continue;
        }
        fence_after();
        if (idx + 1 == W.count) bad |= (S.bad[0][items % kPieces] | S.bad[1][items % kPieces]) != 0;
        if (active) {
          const uint32_t ts = tm + lanes + w * kTile;
          uint32_t sc[H::kChunk];
          auto load = [&](int y) {               // scores y.. of this thread's
            tm_load<H::kChunk>(sc, ts + half * cols + y);
            if (!edge) return;
            const uint64_t see = sv::seen_bits(j0 + half * cols + y - n, tok, mask, par);
            const uint32_t lo = static_cast<uint32_t>(see), hi = static_cast<uint32_t>(see >> 32);
#pragma unroll
            for (int z = 0; z < H::kChunk; ++z)
              if (!(((z < 32 ? lo : hi) >> (z & 31)) & 1)) sc[z] = 0xff800000u;
          };
          float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int y = 0; y < cols; y += H::kChunk) {
            load(y);
#pragma unroll
            for (int z = 0; z < H::kChunk; ++z) v[z & 3] = fmaxf(v[z & 3], __uint_as_float(sc[z]));
          }
          float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
          if (one) {
            S.row_max[x & 1][half][row] = top;
            sv::named_bar_sync(2 + wq, 64);      // the two warps of these rows: both have read their scores
            top = fmaxf(top, S.row_max[x & 1][half ^ 1][row]);
          }
          // The first tile sets the maximum; later ones move it when it has grown by over kSlack.
          const bool grew = top > mx && (mx == -INFINITY || (top - mx) * c > sv::kSlack);
          if (__any_sync(kFull, grew)) {
            const float f = !grew ? 1.0f : (mx == -INFINITY ? 0.0f : sv::ex2((mx - top) * c));
            if (grew) mx = top;
            l *= f;
            if (idx > 0) {                     // the products with the tiles before are done
              const int e = 2 * x - 1;
              wait_unless_lost(sv::smem_addr(S.empty + e % kSlots), (e / kSlots) & 1, lost);
              __syncwarp();
              fence_after();
#pragma unroll 1
              for (int y = 0; y < outs; y += 16) {
                uint32_t o[16];
                tm_load16(o, to + y);
#pragma unroll
                for (int z = 0; z < 16; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * f);
                tm_store16(to + y, o);
              }
            }
          }
          const float m0 = mx == -INFINITY ? 0.0f : mx, b = F16 ? kBits : -m0 * c;
          const sv::f32x2 m2 = sv::pk(m0, m0), c2 = sv::pk(c, c), b2 = sv::pk(b, b);
          sv::f32x2 sum[2] = {sv::pk(0.0f, 0.0f), sv::pk(0.0f, 0.0f)};
#pragma unroll 1
          for (int y = 0; y < cols; y += H::kChunk) {
            if (cols > H::kChunk) load(y);       // read again: all of a row would not fit the registers
            uint32_t p[H::kChunk / 2];
#pragma unroll
            for (int z = 0; z < H::kChunk / 2; ++z) {
              float p0, p1;
              sv::f32x2 s2 = sv::pk(__uint_as_float(sc[2 * z]), __uint_as_float(sc[2 * z + 1]));
              if (F16) s2 = sv::sub2(s2, m2);
              sv::upk(sv::fma2(s2, c2, b2), p0, p1);
              p0 = sv::ex2(p0);
              p1 = sv::ex2(p1);
              sum[z & 1] = sv::add2(sum[z & 1], sv::pk(p0, p1));
              p[z] = sv::pack2<F16>(p0, p1);
            }
            tm_store<H::kChunk / 2>(ts + (half * cols + y) / 2, p);
          }
          float s0, s1;
          sv::upk(sv::add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
          tm_wait_store();
        }
        if (edge) {
          // Value rows of the round's own entries: what is not finite is cleared; rows behind the last
          // entry are cleared whole.
          unsigned char* vb = dyn + s * H::kSlotBytes;
          const int r0 = max(n - j0, 0);
          // (Two ways: the first way's warps, whose product comes first.)
          const int threads = one ? kSoft : kSoft / 2;
          for (int y = r0 * (D / 8) + tid; way == 0 && y < kTile * (D / 8); y += threads) {
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
        if (lane == 0) {
          sv::mbar_arrive(sv::smem_addr(S.p_ready + w));
          if (kOne && !one) sv::mbar_arrive(sv::smem_addr(S.p_ready + w));   // (it counts the warps of one way)
        }
      }
      wait_unless_lost(sv::smem_addr(&S.o_full), items & 1, lost);
      __syncwarp();
      fence_after();
      if (bad || *lost) atomicOr(&S.flags, 1);
      if (odd) atomicOr(&S.flags, 2);
      base += W.count;
      ++items;
      if (!one) used[way ^ 1] += W.count;      // the other way's

      // One way: a row's sum is that of its two threads; each finishes half of the row's columns.
      float* sums = &S.row_max[0][0][0];       // [2][kRows]; the tiles are done with it
      if (one) sums[half * kRows + row] = l;
      sv::named_bar_sync(1, kSoft);
      const int flags = S.flags;
      const float jl = (flags & 1) ? __int_as_float(0x7fffffff) : (one ? sums[row] + sums[kRows + row] : l);
      const bool whole = W.count == W.tiles;
      const int slot = (2 * blockIdx.x + (W.first == 0 ? 1 : 0)) * kWays + way;
      size_t to_row = 0;                       // kShared: the result's row, of a side or a part
      if constexpr (kShared) {
        const int r = row0 + row, i = r / R.group;
        to_row = whole ? P.side_at(side, (static_cast<size_t>(W.token0) + i) * P.Hq + W.head * R.group + r - i * R.group)
                       : static_cast<size_t>(slot) * kRows + row;
      }
      const int i = (row0 + row) / R.group, hq = W.head * R.group + (row0 + row) - i * R.group;
      const size_t at = (static_cast<size_t>(W.row) * R.N + i) * P.Hq + hq;
      const float inv = 1.0f / jl;
#pragma unroll 1
      for (int k = 0; k < outs; k += 16) {
        if (!active) break;
        const int mycol = half * outs + k;
        uint32_t o[16];
        tm_load16(o, to + k);
        float f[16];
#pragma unroll
        for (int z = 0; z < 16; ++z) f[z] = __uint_as_float(o[z]);
        // Values that are not finite were left out of the products, where a zero probability would have
        // made NaN of them: they are added to the rows that attend them.
        if (flags & 2) {
          const int32_t* table = C.table + static_cast<size_t>(W.row) * C.max_pages;
          if constexpr (kShared) {
            sv::SharedWork w;
            sv::row_work(R, W.row, &w);
            table = sv::pages_of(R, W.row, w);
          }
          for (int j = max(n, W.first * kTile); j < min(entries, last * kTile); ++j) {
            const int page = __ldg(table + (j >> C.page_log2)), a = j - n;
            if (!sv::page_ok(C, page)) continue;
            if (!(par ? a <= 0 || ((mask >> (a - 1)) & 1) : a <= tok)) continue;
            const unsigned short* v = reinterpret_cast<const unsigned short*>(C.v + sv::entry_offset(C, page, W.head, j)) + mycol;
#pragma unroll
            for (int z = 0; z < 16; ++z) {
              const float e = sv::value_of<F16>(v[z]);
              if (!isfinite(e)) f[z] += e;
            }
          }
        }
        if (row < rows) {
          if constexpr (kShared) {
            float* out = (whole ? P.side_o : P.part_o) + to_row * D + mycol;
            store8(out, f);
            store8(out + 8, f + 8);
          } else if (whole) {
            uint32_t p[8];
#pragma unroll
            for (int z = 0; z < 8; ++z) p[z] = sv::pack2<F16>(f[2 * z] * inv, f[2 * z + 1] * inv);
            uint4* out = reinterpret_cast<uint4*>(static_cast<char*>(P.out) + (at * D + mycol) * 2);
            out[0] = make_uint4(p[0], p[1], p[2], p[3]);
            out[1] = make_uint4(p[4], p[5], p[6], p[7]);
          } else {
            float* out = P.part_o + (static_cast<size_t>(slot) * D + mycol) * kRows + row;
#pragma unroll
            for (int z = 0; z < 16; ++z) out[z * kRows] = f[z];
          }
        }
      }
      if (half == 0 && row < rows) {
        if constexpr (kShared) (whole ? P.side_ml : P.part_ml)[to_row] = make_float2(mx, jl);
        else if (!whole) P.part_ml[slot * kRows + row] = make_float2(mx, jl);
        else if (P.lse) P.lse[at] = (mx * c + (log2f(jl) - kBits)) * 0.6931471805599453f;
      }
      fence_before();
      sv::named_bar_sync(1, kSoft);            // the sums have been read
      if ((tid & 127) == 0 && half == 0 && W.first == 0 && rows > 0)
        if constexpr (kShared) sv::tell_shared(P, W.row, W.head, W.q_tile * kWays + way, W.tokens, W.token0, whole, W.item_at, W.tiles, S.plan);
        else sv::tell_shared(P, way, W.row, W.head, W.q_tile * kWays + way, rows, whole, W.item_at, W.tiles, S.plan);
    }
    fence_before();
  }
  if constexpr (kShared)
    if (blockIdx.x == 0 && tid == 0) *P.bad_groups = S.plan.bad;
  __syncthreads();
  if (warp == kProducts) {
    if (S.lost && lane == 0) {                 // products in flight end before the tensor memory is given back
      products_done(sv::smem_addr(&S.drained));
      sv::mbar_wait_drain(sv::smem_addr(&S.drained), 0);
    }
    __syncwarp();
    tm_free(tm);
  }
  if (S.lost) {                                // a wait gave up: NaN for the whole run
    sv::WalkOf<kShared> W;
    W.begin(R, S.plan);
    while (W.next(R))
#pragma unroll 1
      for (int way = 0; way < kWays; ++way) {
        const int q_tile = W.q_tile * kWays + way, row0 = q_tile * P.tile_rows;
        const int rows = min(P.tile_rows, sv::tokens_of(W.w) * R.group - row0);
        const bool whole = W.count == W.w.tiles;
        const int slot = (2 * blockIdx.x + (W.first == 0 ? 1 : 0)) * kWays + way;
        int token0 = 0, side = 0;
        if constexpr (kShared) {
          token0 = W.w.token0;
          side = W.row >= R.groups;
        }
#pragma unroll 1
        for (int x = tid; x < rows * D; x += kThreads) {
          const int r = x / D, i = (row0 + r) / R.group, hq = W.head * R.group + (row0 + r) - i * R.group;
          const size_t at = ((kShared ? static_cast<size_t>(token0) : static_cast<size_t>(W.row) * R.N) + i) * P.Hq + hq;
          if constexpr (kShared) {
            if (x % D == 0 && whole) P.side_ml[P.side_at(side, at)].y = __int_as_float(0x7fffffff);
          } else {
            if (whole) static_cast<unsigned short*>(P.out)[at * D + x % D] = 0x7fffu;
            if (x % D == 0 && whole && P.lse) P.lse[at] = __int_as_float(0x7fffffff);
          }
          if (x % D == 0 && !whole) P.part_ml[static_cast<size_t>(slot) * kRows + r].y = __int_as_float(0x7fffffff);
        }
        if (tid == 0 && W.first == 0 && rows > 0) {
          if constexpr (kShared) sv::tell_shared(P, W.row, W.head, q_tile, sv::tokens_of(W.w), token0, whole, W.item_at, W.w.tiles, S.plan);
          else sv::tell_shared(P, way, W.row, W.head, q_tile, rows, whole, W.item_at, W.w.tiles, S.plan);
        }
      }
  }
}

template <bool F16, int D, int kWays, bool kShared>
int launch(const ParamsOf<kShared>& P, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q, int q_tokens,
           int grid, cudaStream_t st) {
  static_assert(kSmemBytes<D, kWays> <= 232448, "shared memory");
  auto kern = sv_attend_wide_kernel<F16, D, kWays, kShared>;
  static std::atomic<unsigned long long> allowed{0};
  if (sv::allow_shared(kern, (kSmemBytes<D, kWays>), allowed) != SV_OK) return SV_ERR_CUDA;
  if constexpr (kShared)
    if (P.R.first) return sv::launch_ahead(kern, dim3(grid), kThreads, kSmemBytes<D, kWays>, st, P, k, v, q, q_tokens);
  kern<<<grid, kThreads, (kSmemBytes<D, kWays>), st>>>(P, k, v, q, q_tokens);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

template <bool F16, bool kShared>
int launch_type(const ParamsOf<kShared>& P, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q, int q_tokens,
                int grid, cudaStream_t st) {
  const int D = P.R.C.head_dim;
  if (D == 256) return launch<F16, 256, 1, kShared>(P, k, v, q, q_tokens, grid, st);
  if (D == 128)
    return P.ways == 2 ? launch<F16, 128, 2, kShared>(P, k, v, q, q_tokens, grid, st)
                       : launch<F16, 128, 1, kShared>(P, k, v, q, q_tokens, grid, st);
  return P.ways == 2 ? launch<F16, 64, 2, kShared>(P, k, v, q, q_tokens, grid, st)
                     : launch<F16, 64, 1, kShared>(P, k, v, q, q_tokens, grid, st);
}

}  // namespace
