// What the attention and weight kernels share: the split of a batch's key tiles over the CTAs, the
// copies of a tile from the pages, and the matrix instructions.
#pragma once

#include "sv_cache.cuh"
#include "sv_common.cuh"

namespace sv {

// The round a batch is in, and how its work divides. A row's work is one item per key head and tile of
// query rows (row r = token r / group, query head r % group of the key head's); an item is
// ceil((n + m) / tile) key tiles. The batch's work in units of a tile, in the order (row, head, query
// tile, key tile), each item's tiles preceded by `extra` units for its queries and its end, is cut into
// equal runs, one per CTA: no CTA gets over one unit more than another, whatever the lengths are, and
// only the items at a run's ends are shared with another CTA.
struct Round {
  Cache C;
  const int32_t* prefix;
  const int32_t* num;
  int B, N, group, q_rows;                // q_rows: query rows of a query tile
  int tile_log2;                          // entries of a key tile
  int extra;                              // what an item costs besides its tiles, in tiles
  bool none_ok;                           // num = -1 counts as no token
};

struct RowWork {
  int n, m, tiles, q_tiles;
};

// False for a row in error (no work).
__device__ __forceinline__ bool row_work(const Round& R, int b, RowWork* w) {
  const bool ok = round_lengths(R.C, R.prefix, R.num, b, R.N, R.none_ok, &w->n, &w->m);
  const bool some = ok && w->m > 0;
  w->tiles = some ? (w->n + w->m + (1 << R.tile_log2) - 1) >> R.tile_log2 : 0;
  w->q_tiles = some ? (w->m * R.group + R.q_rows - 1) / R.q_rows : 0;
  return ok;
}
__device__ __forceinline__ long long row_units(const Round& R, const RowWork& w) {
  return static_cast<long long>(w.tiles + R.extra) * w.q_tiles * R.C.heads;
}

struct Plan {
  long long total;                        // units of the batch
  long long parts;                        // CTAs with work: each of them has a unit at least
  long long at;                           // first unit of this CTA's run
  long long row_at;                       // first unit of the row that holds it
  int row;
};

// Where this CTA's run begins; every thread of the CTA calls it (kThreads of them), `sh` and `plan` in
// shared memory.
template <int kThreads>
__device__ void make_plan(const Round& R, long long (&sh)[kThreads / 32], Plan* plan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (R.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, R.B), b1 = min(b0 + per, R.B);
  long long sum = 0;
  RowWork w;
  for (int b = b0; b < b1; ++b) {
    row_work(R, b, &w);
    sum += row_units(R, w);
  }
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  long long before = incl - sum, total = 0;
#pragma unroll
  for (int x = 0; x < kThreads / 32; ++x) {
    if (x < warp) before += sh[x];
    total += sh[x];
  }
  const long long parts = total < gridDim.x ? total : gridDim.x;
  const long long at = blockIdx.x < parts ? total * blockIdx.x / parts : total;
  if (tid == 0) {
    plan->total = total;
    plan->parts = parts;
    plan->at = at;
    plan->row = R.B;
  }
  __syncthreads();
  if (at >= before && at < before + sum) {
    long long run = before;
    for (int b = b0; b < b1; ++b) {
      row_work(R, b, &w);
      const long long t = row_units(R, w);
      if (at < run + t) {
        plan->row = b;
        plan->row_at = run;
        break;
      }
      run += t;
    }
  }
  __syncthreads();
}

// The CTA that holds unit t of the batch.
__device__ __forceinline__ int unit_owner(long long t, const Plan& p) {
  return static_cast<int>(((t + 1) * p.parts - 1) / p.total);
}

// A walk over the items of this CTA's run: begin(), then next() while it returns true.
struct Walk {
  long long at, end, row_at, item_at;     // item_at: the unit of the item's first tile
  int row, head, q_tile, first, count;    // key tiles [first, first + count) of the item
  RowWork w;

  __device__ __forceinline__ void begin(const Round& R, const Plan& p) {
    at = p.at;
    end = blockIdx.x < p.parts ? p.total * (blockIdx.x + 1) / p.parts : at;
    row = p.row;
    row_at = p.row_at;
    if (at < end) row_work(R, row, &w);
  }
  __device__ __forceinline__ bool next(const Round& R) {
    do {
      if (at >= end) return false;
      while (at - row_at >= row_units(R, w)) {     // past this row: the next one with work
        row_at += row_units(R, w);
        ++row;
        row_work(R, row, &w);
      }
      const int per = w.tiles + R.extra;
      const int in_row = static_cast<int>(at - row_at), item = in_row / per, in_item = in_row - item * per;
      head = item / w.q_tiles;
      q_tile = item - head * w.q_tiles;
      item_at = at - in_item + R.extra;
      const int stop = end - at < per - in_item ? in_item + static_cast<int>(end - at) : per;
      first = in_item > R.extra ? in_item - R.extra : 0;
      count = stop - R.extra - first;
      at += stop - in_item;
    } while (count <= 0);                 // the run ended before the item's first tile
    return true;
  }
};

// ------------------------------------------------------------------------------------------------
// Copies
// ------------------------------------------------------------------------------------------------

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int slot,
                                         int head, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(map), "r"(x), "r"(slot), "r"(head), "r"(page), "r"(bar)
      : "memory");
}

// The page numbers of a tile's boxes for lane `lane` of the producer warp: box x of an array covers
// `rows` entries of one page and 64 of the D elements. Lanes take (array, box, 64 elements) in order.
struct TileLoader {
  int boxes_log2, halves_log2, rows_log2, tile_log2, ops;

  __device__ __forceinline__ void init(const Cache& C, int arrays, int log2_entries) {
    tile_log2 = log2_entries;
    rows_log2 = C.page_log2 < 6 ? C.page_log2 : 6;
    boxes_log2 = tile_log2 - rows_log2;
    halves_log2 = C.head_dim == 64 ? 0 : (C.head_dim == 128 ? 1 : 2);
    ops = arrays << (boxes_log2 + halves_log2);
  }
  // Whether operation `op` of a tile copies entries of the row, and the page number it then has (unchecked: a
  // use of the number waits for its load).
  __device__ __forceinline__ bool has(int tile, int entries, int op) const {
    const int box = (op >> halves_log2) & ((1 << boxes_log2) - 1);
    return op < ops && (tile << tile_log2) + (box << rows_log2) < entries;
  }
  __device__ __forceinline__ int page(const Cache& C, int row, int tile, int op) const {
    const int box = (op >> halves_log2) & ((1 << boxes_log2) - 1);
    return cache_page(C, row, (tile << tile_log2) + (box << rows_log2));
  }
  // The copy of operation `op`: stage holds the arrays one after the other, each [D / 64][tile][64].
  __device__ __forceinline__ void load(const Cache& C, const CUtensorMap* k, const CUtensorMap* v,
                                       int tile, int head, int p, int op, uint32_t stage,
                                       uint32_t bar) const {
    const int half = op & ((1 << halves_log2) - 1);
    const int box = (op >> halves_log2) & ((1 << boxes_log2) - 1);
    const int array = op >> (halves_log2 + boxes_log2);
    const int j = (tile << tile_log2) + (box << rows_log2);
    const uint32_t dst = stage + (((array << halves_log2) + half) << (tile_log2 + 7)) + (box << (rows_log2 + 7));
    tma_load(dst, array ? v : k, half * 64, j & (C.page_size - 1), head, p, bar);
  }
};

// A lane's pages of the tiles of a run, read kPagesAhead tiles before the copies that need them: a load
// takes about as long as a tile while the cache streams (one tile ahead, a tile took 0.85 us whatever its size).
constexpr int kPagesAhead = 4;
struct PagesAhead {
  int p[kPagesAhead];

  __device__ __forceinline__ void begin(const TileLoader& T, const Cache& C, int row, int first, int last,
                                        int entries, int op) {
#pragma unroll
    for (int x = 0; x < kPagesAhead; ++x)
      p[x] = first + x < last && T.has(first + x, entries, op) ? T.page(C, row, first + x, op) : 0;
  }
  // The page of `tile`: -1 where the operation copies nothing, -2 when it is out of range. Reads that of
  // tile + kPagesAhead.
  __device__ __forceinline__ int next(const TileLoader& T, const Cache& C, int row, int tile, int last,
                                      int entries, int op) {
    const int now = p[0], ahead = tile + kPagesAhead;
#pragma unroll
    for (int x = 0; x + 1 < kPagesAhead; ++x) p[x] = p[x + 1];
    p[kPagesAhead - 1] = ahead < last && T.has(ahead, entries, op) ? T.page(C, row, ahead, op) : 0;
    return !T.has(tile, entries, op) ? -1 : (page_ok(C, now) ? now : -2);
  }
};

// ------------------------------------------------------------------------------------------------
// Matrix instructions and their operands in shared memory (rows of 128 bytes, 16-byte chunks swizzled
// by the row's low three bits as the tensor maps write them)
// ------------------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t swizzled(uint32_t base, int row, int chunk) {
  return base + row * 128 + ((chunk ^ (row & 7)) << 4);
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two fp32 values rounded to the cache's type, lo in the low half.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ------------------------------------------------------------------------------------------------
// Which of the round's tokens a token attends
// ------------------------------------------------------------------------------------------------

// Per token of a tree the tokens 1..64 that it attends (its ancestors and itself; all attend token 0),
// as bits 0..63. Called by `threads` threads, thread `tid`; returns whether this thread's nodes are
// valid. A walk upwards ends: it stops at a parent that is not below its node.
__device__ __forceinline__ bool tree_masks(const int32_t* parents, int m, unsigned long long* masks,
                                           int tid, int threads) {
  bool ok = true;
  for (int t = tid; t < m; t += threads) {
    const int p = __ldg(parents + t);
    ok &= t == 0 ? p == -1 : (p >= 0 && p < t);
    unsigned long long s = 0;
    for (int x = t; x > 0;) {
      s |= 1ull << (x - 1);
      const int up = __ldg(parents + x);
      if (up >= x) break;
      x = up;
    }
    masks[t] = s;
  }
  return ok;
}

// The same of one token t.
__device__ __forceinline__ unsigned long long tree_mask(const int32_t* parents, int t) {
  unsigned long long s = 0;
  for (int x = t; x > 0;) {
    s |= 1ull << (x - 1);
    const int up = __ldg(parents + x);
    if (up >= x) break;
    x = up;
  }
  return s;
}

// Which of 64 entries a token attends, as bits: a0 is the place in the round of the first of them (below
// 0: an entry before the round), i the token; in a tree `mask` is the token's from tree_masks.
__device__ __forceinline__ uint64_t seen_bits(int a0, int i, unsigned long long mask, bool tree) {
  const int all = (tree ? 0 : i) - a0 + 1;       // places up to this one are attended: token 0's, or i's
  uint64_t s = all >= 64 ? ~0ull : (all > 0 ? (1ull << all) - 1 : 0ull);
  if (tree) {                                    // place a >= 1 is bit a - 1 of the mask
    if (a0 <= 0) s |= 1 - a0 < 64 ? mask << (1 - a0) : 0ull;
    else s = a0 - 1 < 64 ? mask >> (a0 - 1) : 0ull;
  }
  return s;
}

}  // namespace sv
