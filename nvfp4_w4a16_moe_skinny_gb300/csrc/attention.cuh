// Attention over a paged cache, few rows at a time: decode steps, verify blocks
// and short chunks (paged_attention); and what both attention kernels share.
//
// One pass over the keys.  With the running maximum m of a row's logits s_j (in units of log 2),
//   l = sum_j 2^(s_j - m),   o = sum_j 2^(s_j - m) v_j,   out = o / l,   lse = (m + log2 l) ln 2,
// and when m grows, l and o are multiplied by 2^(m_old - m).  Sums over disjoint keys join the same way.
//
// Rows.  The heads of one kv head and the new tokens of one sequence are packed
// into rows r = token * group + head, so the keys and values of a kv head are
// read once for all of them; a row tile is 16 * RW of these rows.
//
// Split.  An item is (sequence, row tile, kv head); its keys are cut into units
// of kKeys keys.  All units, numbered item by item, are dealt to the grid in contiguous
// ranges of equal length, so ragged lengths balance by themselves and a single long sequence
// fills the chip.  Every CTA finds its range from kv_len and cu_tokens by itself (a block-wide
// scan), so one launch geometry serves a captured graph at any lengths.  An item that lies in one range is
// finished in registers; otherwise its holders write their shares (o, m and l, fp32) to the
// workspace, at most two per CTA, and a second grid joins them in range order: the
// result does not depend on timing, and no CTA waits for another.
//
// Inner loop.  One producer warp copies K and V tiles by TMA (swizzled boxes of a
// page's rows; a page id outside the pool is an out-of-range coordinate, which
// reads as zeros and touches no memory) into a ring of stages; four
// consumer warps run m16n8k16 MMAs.  RW warps share a key slice and split the rows,
// KW = 4 / RW key slices share the rows: a decode step (one row tile of 16) has four
// slices, each with its own running maximum and sum, joined through shared memory once per
// item; no barrier stops the loop between tiles.  Q lies in shared memory and comes by ldmatrix like K, so that
// registers suffice for two CTAs an SM.
//
// Numbers.  bf16 caches: bf16 products, fp32 sums, weights rounded to bf16 (half a
// step of 2^-8, as the result itself).  E4M3 caches: codes convert to f16 exactly;
// q is scaled by a power of two per row into f16's range (exact down to 2^-31
// of the row's largest value) and weights are scaled by 2^15 before their rounding to f16 (2^-11).
//
// What bounds it.  Memory, where the keys are many: 64 sequences of up to 16K keys (32 heads on 8
// kv heads of 128 bf16 values, 520 MB) take 89 us, 85% of the rate of a plain copy, two
// of 131,071 keys over an E4M3 cache (537 MB) 90 us, 88%.  The chain of two launches, the search for the
// range, the first page look-ups and copies and the join elsewhere: one sequence of 1,000 keys 9.4 us.
// A row tile is too thin for tcgen05: its products take 128 rows at a time, and the same time for 16.
#pragma once

#include <type_traits>

#include "launch.cuh"
#include "paged.cuh"

namespace nvfp4 {

constexpr size_t kAttnCounterBytes = 4096;  // at the start of the workspace
constexpr size_t kAttnSplitBytes = 8192;    // after them: a split_item of every CTA of the split kernel
constexpr int kAttnGrid = 152;  // SMs that the split is made for; fixed, so that workspace sizes are host-computable

// Division by a number that a launch knows: x / g = umulhi(x, mul) >> shift for
// x < 2^31 (shift < 0: g = 1).
struct FastDiv {
  uint32_t mul;
  int shift;
};

inline FastDiv fast_div(int g) {
  if (g == 1) return {0, -1};
  int s = 0;
  while ((int64_t{1} << s) < g) ++s;
  return {static_cast<uint32_t>(((uint64_t{1} << (31 + s)) + g - 1) / g), s - 1};
}

struct AttnJob {
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* table;
  int n_seqs, max_pages, n_tokens;
  int n_heads, n_kv, group;
  FastDiv by_group;
  int page_log2, num_pages;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  int64_t out_stride;
  float* lse;
  const void* v_pool;
  int64_t page_stride;
  const float* k_scale;
  const float* v_scale;
  float scale, softcap;
  int window;
  unsigned* counters;  // arrivals at the join of each split item, by the range that holds its start
  float* part;         // shares: unnormalised sums, reference maxima and sums of weights of a row tile, two per CTA
  int4* split;         // the split kernel's split items, by the range that holds their start (split_item)
  const uint32_t* masks;  // tree_attention: which new tokens each new token sees, mask_words 32-bit words a token
  int mask_words;
};

struct KvMaps {
  CUtensorMap k, v;
};

// ------------------------------------------------------------------ work decomposition

// What the kernels and the host-side check of the split (paged_attention_plan_check) share is
// compiled for both.
//
// Tiling of one kernel: rows of a row tile, keys of a unit, and what starting and
// finishing an item counts for, in units (the ranges are balanced with it).
// `snap`: a range boundary that falls this close to an item's end moves there, so that no
// item is split for a few units.
// `least`: a call of fewer units than this for each CTA takes one range for every `least` units
// or part of them, equal ones, so that a range may hold a little less (nine units by fours: three ranges
// of three).
// What they are worth is measured at AttnTile and ChunkTile.
struct Tiling {
  int rows, keys, over, snap, least;
};

// The tiling of a tree_attention call: a token sees all keys before the new ones and, of those, what
// its mask says.  (A type of its own, so that the causal kernels compile as if there were no trees: a
// member that says it cost them registers, 16 sequences of 8,000 keys with 64 rows 130 us instead of 127.)
struct TreeTiling : Tiling {};
template <typename G>
constexpr bool kIsTree = std::is_same_v<G, TreeTiling>;
template <bool kTree>
__host__ __device__ constexpr auto tiling_for(const Tiling& t) {
  if constexpr (kTree)
    return TreeTiling{t};
  else
    return t;
}

// Quotient of x < 2^31 by the divisor that `d` was made for (fast_div): a multiply by the
// rounded-up reciprocal and a shift.
__host__ __device__ __forceinline__ int div_by(const FastDiv d, int x) {
#ifdef __CUDA_ARCH__
  return d.shift < 0 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), d.mul) >> d.shift);
#else
  const uint64_t product = static_cast<uint64_t>(static_cast<uint32_t>(x)) * d.mul;
  return d.shift < 0 ? x : static_cast<int>(static_cast<uint32_t>(product >> 32) >> d.shift);
#endif
}

struct Sequence {
  int tok0, n, len, rows, tiles;
};

// From cu_tokens[b], cu_tokens[b + 1] and kv_len[b].
__host__ __device__ __forceinline__ Sequence sequence_from(const AttnJob& p, int lo, int hi, int len, const Tiling& g) {
  Sequence s;
  s.tok0 = min(max(lo, 0), p.n_tokens);
  s.n = min(max(hi, s.tok0), p.n_tokens) - s.tok0;
  s.len = min(max(len, 0), p.max_pages << p.page_log2);
  s.rows = s.n * p.group;
  s.tiles = (s.rows + g.rows - 1) / g.rows;
  return s;
}
__device__ __forceinline__ Sequence sequence_of(const AttnJob& p, int b, const Tiling& g) {
  return sequence_from(p, __ldg(p.cu + b), __ldg(p.cu + b + 1), __ldg(p.kv_len + b), g);
}

// A row tile of one sequence and the keys that any of its rows sees, [lo, hi).
struct RowTile {
  int row0, rows;    // first packed row and number of rows
  int lo, hi;
  int tile0, units;  // first key tile, number of units (at least one, so that empty rows are written)
};

template <typename G>
__host__ __device__ __forceinline__ RowTile row_tile(const AttnJob& p, const Sequence& s, int rt, const G& g) {
  RowTile t;
  t.row0 = rt * g.rows;
  t.rows = min(g.rows, s.rows - t.row0);
  if constexpr (kIsTree<G>) {  // (a row whose mask is empty sees the context's last keys)
    t.hi = s.len;
    t.lo = p.window > 0 ? min(max(max(s.len - s.n, 0) - p.window, 0), t.hi) : 0;
  } else {
    const int p0 = s.len - s.n + div_by(p.by_group, t.row0);
    const int p1 = s.len - s.n + div_by(p.by_group, t.row0 + t.rows - 1);
    t.hi = min(max(p1 + 1, 0), s.len);
    t.lo = p.window > 0 ? min(max(p0 - p.window + 1, 0), t.hi) : 0;
  }
  t.tile0 = t.lo / g.keys;
  t.units = max(1, (t.hi + g.keys - 1) / g.keys - t.tile0);
  return t;
}

// Units of `s`, overheads included, by one lane or (lane, step) by the lanes of a warp.
template <typename G>
__device__ __forceinline__ long long tile_units(const AttnJob& p, const Sequence& s, int first, int step, const G& g) {
  long long u = 0;
#pragma unroll 1
  for (int rt = first; rt < s.tiles; rt += step) u += row_tile(p, s, rt, g).units + g.over;
  return u * p.n_kv;
}

// The split of all units into contiguous ranges, one per CTA.
struct Ranges {
  long long total, each;
  int grid, more;  // ranges in use; the first `more` of them hold each + 1 units
  __host__ __device__ __forceinline__ void set(long long all, int ctas, int least) {
    total = all;
    grid = all >= static_cast<long long>(ctas) * least ? ctas : (static_cast<int>(all) + least - 1) / least;
    if (grid < 1) {
      each = more = 0;
    } else if (all >> 31) {
      each = all / grid;
      more = static_cast<int>(all - each * grid);
    } else {
      const uint32_t q = static_cast<uint32_t>(all) / static_cast<uint32_t>(grid);
      each = q;
      more = static_cast<int>(static_cast<uint32_t>(all) - q * grid);
    }
  }
  __host__ __device__ __forceinline__ long long start(int c) const { return c * each + min(c, more); }
  __host__ __device__ __forceinline__ int holder(long long u) const {
    const long long cut = more * (each + 1), by = u < cut ? each + 1 : each, at = u < cut ? u : u - cut;
    const int before = u < cut ? 0 : more;
    if (total >> 31) return before + static_cast<int>(at / by);
    return before + static_cast<int>(static_cast<uint32_t>(at) / static_cast<uint32_t>(by));
  }
};

// Where a CTA starts: the sequence that holds its first unit, and the units before it.
struct Found {
  int seq;
  long long before;
};

// What find_range keeps in shared memory.
struct RangeScratch {
  long long warp_sum[32], before;
  int seq, n_long;
};

// Block-wide scan of the sequences' units (every thread of the block calls it).  Sets the
// ranges and, if range c is in use, finds where its first unit lies.  A thread sums its
// sequence's row tiles itself if they are few; long sequences go through a list (kList
// entries of scratch memory) to whole warps.
template <int kThreadsInBlock, typename G>
__device__ __forceinline__ void find_range(const AttnJob& p, const G& g, int ctas, int c, Ranges* ranges,
                                           Found* found, RangeScratch* sh, longlong2* list) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kNW = kThreadsInBlock / 32;
  long long mine = 0, incl = 0;
  if (p.n_seqs <= 32) {  // few sequences, few of them long: every warp finds the same by itself
    Sequence s{};
    if (lane < p.n_seqs) s = sequence_of(p, lane, g);
    unsigned longs = __ballot_sync(0xffffffffu, s.tiles > 4);
    if (__popc(longs) <= 2) {
      mine = s.tiles > 4 ? 0 : tile_units(p, s, 0, 1, g);
      for (; longs; longs &= longs - 1) {
        const int who = __ffs(longs) - 1;
        Sequence o;
        o.n = __shfl_sync(0xffffffffu, s.n, who), o.len = __shfl_sync(0xffffffffu, s.len, who);
        o.rows = __shfl_sync(0xffffffffu, s.rows, who), o.tiles = __shfl_sync(0xffffffffu, s.tiles, who);
        long long part = tile_units(p, o, lane, 32, g);
#pragma unroll 1
        for (int d = 16; d > 0; d >>= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
        if (lane == who) mine = part;
      }
      incl = mine;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      ranges->set(__shfl_sync(0xffffffffu, incl, 31), ctas, g.least);
      const long long u = ranges->start(c);
      const unsigned here = __ballot_sync(0xffffffffu, u >= incl - mine && u < incl);
      found->seq = here ? __ffs(here) - 1 : 0;
      found->before = __shfl_sync(0xffffffffu, incl - mine, found->seq);
      return;
    }
  }
  // one pass for the total, then (again over the batch only where it is longer than
  // the block) one that finds the unit
  const bool once = p.n_seqs <= kThreadsInBlock;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    long long base = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.n_seqs; b0 += kThreadsInBlock) {
      if (pass == 0 || !once) {
        const int b = b0 + threadIdx.x;
        Sequence s{};
        if (b < p.n_seqs) s = sequence_of(p, b, g);
        const bool is_long = s.tiles > 4;
        mine = is_long ? 0 : tile_units(p, s, 0, 1, g);
        if (threadIdx.x == 0) sh->n_long = 0;
        if (__syncthreads_or(is_long)) {
          int at = 0;
          if (is_long) {
            at = atomicAdd(&sh->n_long, 1);
            list[at].x = b;
          }
          __syncthreads();
          for (int i = warp; i < sh->n_long; i += kNW) {
            long long part = tile_units(p, sequence_of(p, static_cast<int>(list[i].x), g), lane, 32, g);
#pragma unroll 1
            for (int d = 16; d > 0; d >>= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
            if (lane == 0) list[i].y = part;
          }
          __syncthreads();
          if (is_long) mine = list[at].y;
        }
        incl = mine;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        if (lane == 31) sh->warp_sum[warp] = incl;
        __syncthreads();
        long long pre = base;
#pragma unroll 1
        for (int w = 0; w < kNW; ++w) {
          const long long v = sh->warp_sum[w];
          if (w < warp) pre += v;
          base += v;
        }
        incl += pre;
      }
      if (pass == 1) {
        const long long u = ranges->start(c);
        if (mine > 0 && u >= incl - mine && u < incl) {
          sh->seq = b0 + threadIdx.x;
          sh->before = incl - mine;
        }
      }
      __syncthreads();
    }
    if (pass == 0) {
      ranges->set(base, ctas, g.least);
      if (c >= ranges->grid) return;
    }
  }
  found->seq = sh->seq;
  found->before = sh->before;
}

// A place in the list of items (sequence, row tile, kv head).  All roles of a CTA walk
// the same list.
struct Walk {
  int b, rt, h;
  long long item0;  // first unit of the item
  Sequence s;
  RowTile t;
};

template <typename G>
__device__ __forceinline__ void walk_seq(const AttnJob& p, Walk& w, const G& g) {
  w.s = sequence_of(p, w.b, g);
  w.rt = 0, w.h = 0;
  if (w.s.tiles > 0) w.t = row_tile(p, w.s, 0, g);
}

// The item that holds unit u, searched from where the walk is; u is below the total.
// All lanes of a warp call it with the same arguments.
template <typename G>
__device__ __forceinline__ void walk_to(const AttnJob& p, Walk& w, long long u, const G& g) {
  const int lane = threadIdx.x & 31;
  while (true) {
    if (w.rt < w.s.tiles) {
      const int span = w.t.units + g.over;
      // one after the other in the usual case; far jumps (a CTA's first item) by division
      if (u < w.item0 + span) return;
      if (w.h + 1 < p.n_kv && u < w.item0 + 2 * static_cast<long long>(span)) {
        w.item0 += span, ++w.h;
        return;
      }
      const long long all = static_cast<long long>(span) * (p.n_kv - w.h);
      if (u < w.item0 + all) {
        const int k = all >> 32 ? static_cast<int>((u - w.item0) / span)
                                : static_cast<int>(static_cast<uint32_t>(u - w.item0) / static_cast<uint32_t>(span));
        w.h += k;
        w.item0 += static_cast<long long>(k) * span;
        return;
      }
      w.item0 += all;
      w.h = 0;
      // the next row tiles, 32 at a time: the first one that ends past u
      int rt = w.rt + 1;
      bool here = false;
#pragma unroll 1
      while (rt < w.s.tiles && !here) {
        const bool in = rt + lane < w.s.tiles;
        const long long mine = in ? static_cast<long long>(row_tile(p, w.s, rt + lane, g).units + g.over) * p.n_kv : 0;
        long long incl = mine;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, in && u < w.item0 + incl);
        const int who = past ? __ffs(past) - 1 : 31;
        const long long before = __shfl_sync(0xffffffffu, incl - mine, who);
        const long long end = __shfl_sync(0xffffffffu, incl, 31);
        here = past != 0;
        w.item0 += here ? before : end;
        rt += here ? who : 32;
      }
      w.rt = here ? rt : w.s.tiles;
      if (here) w.t = row_tile(p, w.s, w.rt, g);
    } else {
      if (++w.b >= p.n_seqs) return;  // not reached for a unit below the total
      walk_seq(p, w, g);
    }
  }
}

// Where a range boundary d units into an item of `units` tiles lies after snapping: 0, the
// whole span, or d.
__host__ __device__ __forceinline__ int snapped(int d, int units, const Tiling& g) {
  const int span = units + g.over, t = min(g.snap, (span - 1) / 2);
  return d <= t ? 0 : (d >= span - t ? span : d);
}

// The share of the walk's item that range [u0, u1) of CTA c holds, from unit u on: key tiles
// [first, first + n) (none, if only the item's overhead falls into the range, or if the
// boundary has moved), and where an unfinished share goes.
struct Share {
  int first, n, slot;
  bool whole;
  long long end;
};

__host__ __device__ __forceinline__ Share share_at(const Walk& w, long long u, long long u0, long long u1, int c,
                                          const Tiling& g) {
  Share q;
  const int units = w.t.units, span = units + g.over;
  const int from = u == u0 ? snapped(static_cast<int>(u - w.item0), units, g) : 0;
  const int to = u1 < w.item0 + span ? snapped(static_cast<int>(u1 - w.item0), units, g) : span;
  q.end = min(w.item0 + span, u1);
  q.n = max(0, min(units, to) - from);
  q.first = w.t.tile0 + from;
  q.whole = q.n == units;
  q.slot = 2 * c + (from > 0 ? 0 : 1);  // a range starts inside at most one item and ends inside one
  return q;
}

// The ranges [c0, c1] that hold tiles of an item (c0 != c1: it is split).
struct Holders {
  int c0, c1;
};
__host__ __device__ __forceinline__ Holders holders_of(const Walk& w, const Ranges& r, const Tiling& g) {
  const int span = w.t.units + g.over, t = min(g.snap, (span - 1) / 2);
  Holders h;
  h.c0 = r.holder(w.item0 + t);  // boundaries up to t units in have moved to the item's start
  h.c1 = max(h.c0, r.holder(w.item0 + min(w.t.units, span - t) - 1));
  return h;
}

// What the join needs of a split item, written by the CTA whose range holds its start: the
// last range that holds a share and the rows (nine bits each; seven are enough for the split kernel's rows), the
// kv head, the first packed row, the sequence's first token.
__device__ __forceinline__ int4 split_item(const Walk& w, int c1) {
  static_assert(2 * kAttnGrid <= 512, "nine bits");
  return make_int4(c1 | w.t.rows << 9, w.h, w.t.row0, w.s.tok0);
}

// ------------------------------------------------------------------ trees

// Bits [0, n) of a word.
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1); }

// What a new token of a tree sees: keys [lo, ctx) of the context, and new token t (key ctx + t) where bit
// t of its mask is set, t >= from.  With a window those are the last of the keys that the mask leaves.
struct TreeRow {
  const uint32_t* mask;
  uint32_t head[2];  // the first two words
  int words, ctx, n, lo, from;
  __device__ __forceinline__ uint32_t word(int i) const {
    if (static_cast<unsigned>(i) < 2u) return i == 0 ? head[0] : head[1];
    return static_cast<unsigned>(i) < static_cast<unsigned>(words) ? __ldg(mask + i) : 0u;
  }
  // keys [key0, key0 + 32), a bit each
  __device__ __forceinline__ uint32_t bits(int key0) const {
    uint32_t m = bits_below(ctx - key0) & ~bits_below(lo - key0);
    const int t0 = key0 - ctx;
    if (t0 > -32)
      m |= __funnelshift_r(word(t0 >> 5), word((t0 >> 5) + 1), t0 & 31) & bits_below(n - t0) & ~bits_below(from - t0);
    return m;
  }
  __device__ __forceinline__ bool sees(int key) const { return bits(key) & 1; }
};

__device__ __forceinline__ TreeRow tree_row(const AttnJob& p, const Sequence& s, int tok) {
  TreeRow r;
  r.mask = p.masks + static_cast<int64_t>(s.tok0 + tok) * p.mask_words;
  r.head[0] = __ldg(r.mask), r.head[1] = __ldg(r.mask + 1);
  r.words = p.mask_words, r.ctx = s.len - s.n, r.n = s.n;
  r.lo = 0, r.from = max(0, -r.ctx);
  if (p.window > 0) {
    int all = 0;
#pragma unroll 1
    for (int t = 0; t < r.n; t += 32) all += __popc(r.word(t >> 5) & bits_below(r.n - t) & ~bits_below(r.from - t));
    r.lo = max(r.ctx, 0) + all - p.window;
#pragma unroll 1
    for (int t = 0; all > p.window; t += 32) {  // the first ones fall out of the window
      uint32_t v = r.word(t >> 5) & bits_below(r.n - t) & ~bits_below(r.from - t);
#pragma unroll 1
      for (; v && all > p.window; v &= v - 1) r.from = t + __ffs(v), --all;
    }
  }
  return r;
}

// ------------------------------------------------------------------ MMA helpers

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool kF16>
__device__ __forceinline__ void mma_16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    mma_f16(c, a, b0, b1);
  else
    mma_bf16(c, a, b0, b1);
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Two E4M3 codes (low, high half of w) -> f16x2, exact.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// tanh(x) for |x| < 1/2: x + x^3 P(x^2), P interpolated at Chebyshev nodes (off by 2^-29; with the
// roundings 2^-24).  1 - 2 / (e^2x + 1) loses what it subtracts there, up to 2^-23 / |x| of the result: with a
// softcap of 50 and logits around 1 the log-sum-exp was off by 5e-6.
constexpr float kTanhSmall = 0.5f;
__device__ __forceinline__ float tanh_small(float x) {
  const float z = x * x;
  float p = fmaf(z, -0.00694294f, 0.02147068f);
  p = fmaf(z, p, -0.05393347f);
  p = fmaf(z, p, 0.13333226f);
  p = fmaf(z, p, -0.33333333f);
  return fmaf(x * z, p, x);
}
__device__ __forceinline__ f32x2 tanh_small2(f32x2 x) {
  const auto both = [](float c) { return pack2(c, c); };
  const f32x2 z = mul2(x, x);
  f32x2 p = fma2(z, both(-0.00694294f), both(0.02147068f));
  p = fma2(z, p, both(-0.05393347f));
  p = fma2(z, p, both(0.13333226f));
  p = fma2(z, p, both(-0.33333333f));
  return fma2(mul2(x, z), p, x);
}
__device__ __forceinline__ float tanh_any(float x) {
  return fabsf(x) < kTanhSmall ? tanh_small(x)
                               : 1.0f - __fdividef(2.0f, exp2_approx(x * 2.8853900817779268f) + 1.0f);
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, int c4,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}

// One lane of a converged warp, chosen by the hardware: unlike a lane test it leaves the
// branch uniform, so that descriptors and addresses stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

__host__ __device__ constexpr int log2c(int v) { return v <= 1 ? 0 : 1 + log2c(v / 2); }

// Halves of packed 16-bit values that are infinite or NaN, as a mask of 0xffff.
template <bool kF16>
__device__ __forceinline__ uint32_t nonfinite_mask(uint32_t v) {
  constexpr uint32_t e = kF16 ? 0x7c007c00u : 0x7f807f80u, one = kF16 ? 0x04000400u : 0x00800080u;
  const uint32_t m = ((v & e) + one) & 0x80008000u;  // the exponent is all ones: the carry reaches the sign bit
  return (m >> 15) * 0xffffu;
}

// bf16 values of q for a scale of zero: zeros, and NaN for infinities and NaN (0 * inf is NaN), so
// that the products carry 0 * NaN from both sides into the logits.
__device__ __forceinline__ uint4 zero_or_nan(uint4 v) {
  return make_uint4(nonfinite_mask<false>(v.x), nonfinite_mask<false>(v.y), nonfinite_mask<false>(v.z),
                    nonfinite_mask<false>(v.w));
}

// ------------------------------------------------------------------ tile geometry

// CTAs of the split kernel on one SM.  Two hide more of each other's waits: 64 sequences of up
// to 16K keys 91 us against 107 with one (128 bf16 values), 16 of 8,000 with 64 rows 76 against 90.
// Heads of 256 values have shared memory for one (a stage is 64 KB), and 64 rows of 128 over an
// E4M3 cache registers (16 sequences of 8,000 keys: 82 us against 103 with two, which spill).
__host__ __device__ constexpr int attn_ctas(int dim, bool fp8, int rw) {
  return dim == 256 || (dim == 128 && fp8 && rw == 4) ? 1 : 2;
}

// Keys of one warp's step: few enough that two stages or more fit in a CTA's shared memory and the
// scores in few registers.
__host__ __device__ constexpr int attn_slice(int dim, bool fp8, int kw) {
  if (kw == 1) return dim == 256 || (dim == 128 && !fp8) ? 32 : 64;
  return dim == 256 || (dim == 128 && !fp8) ? 16 : 32;
}

template <int kDim, bool kFp8, int kRW, int kKW>
struct AttnTile {
  static constexpr int kRows = 16 * kRW;
  static constexpr int kCtas = attn_ctas(kDim, kFp8, kRW);
  static constexpr int kSlice = attn_slice(kDim, kFp8, kKW);              // keys of a warp's step
  static constexpr int kKeys = kSlice * kKW;                         // keys of a unit
  static constexpr int kConsumers = kRW * kKW;
  static constexpr int kThreadsAll = (kConsumers + 1) * 32;
  // in units (Tiling).  An item counted as its units alone: 112 us for the 64 ragged sequences
  // above, with three more 87.  Ranges of four units save shares where there is little to do, two
  // sequences of 2,000 keys with 64 rows 23 us against 33 before the join's present form, but cost verify blocks 7%.
  // Boundaries that move (two units) make no difference here.
  static constexpr int kOver = 3, kSnap = 0, kLeast = 1;
  static constexpr __host__ __device__ Tiling tiling() { return {kRows, kKeys, kOver, kSnap, kLeast}; }
  static constexpr int kEl = kFp8 ? 1 : 2;
  static constexpr int kRowB = kDim * kEl < 128 ? kDim * kEl : 128;  // bytes of a row of a block
  static constexpr int kSub = kDim * kEl / kRowB;                    // blocks across a head
  static constexpr uint32_t kSwz = kRowB == 128 ? 0x70 : 0x30;
  static constexpr int kTileB = kKeys * kDim * kEl;                  // K or V of a unit: page pieces of [kSub][rows][kRowB]
  static constexpr int kStageB = 2 * kTileB;
  static constexpr int kQB = kRows * kDim * 2;                       // Q: [kDim / 64][kRows][128 bytes]
  // a quarter (kKW = 4) or half of the columns of each warp's sums, its reference and sum
  static constexpr int kJoinB = kKW > 1 ? kConsumers * 32 * (kDim / 2 / kKW + 4) * 4 : 0;
  static constexpr int kFit = ((kCtas == 1 ? 227 : 113) * 1024 - 1024 - 1024 - kJoinB - kQB) / kStageB;
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageB + kQB + kJoinB + 1024;
  static_assert(kStages >= 2, "ring too shallow");
};

// Keys that every row of an item sees, [all_lo, all_hi), and that some row sees, [any_lo, any_hi).
struct KeyRange {
  int all_lo, all_hi, any_lo, any_hi;
};

template <bool kTree>
__device__ __forceinline__ KeyRange key_range(const AttnJob& p, const Walk& w) {
  KeyRange r;
  if constexpr (kTree) {
    r.all_hi = max(w.s.len - w.s.n, 0);
    r.all_lo = p.window > 0 ? r.all_hi + w.s.n - p.window : 0;  // (a mask holds n tokens at most)
    r.any_hi = w.t.hi;
    r.any_lo = w.t.lo;
    return r;
  }
  const int first = w.s.len - w.s.n + div_by(p.by_group, w.t.row0);
  const int last = w.s.len - w.s.n + div_by(p.by_group, w.t.row0 + w.t.rows - 1);
  r.all_hi = min(first + 1, w.s.len);
  r.all_lo = p.window > 0 ? last - p.window + 1 : 0;
  r.any_hi = w.t.hi;
  r.any_lo = w.t.lo;
  return r;
}

__device__ __forceinline__ bool partly_seen(const KeyRange& r, int key0, int keys) {
  return key0 + keys > r.all_hi || key0 < r.all_lo;
}

// One 16-byte chunk of V of a key (eight 16-bit values): nothing if no row sees it, and
// without infinities and NaN.
template <bool kF16>
__device__ __forceinline__ uint4 clean_chunk(uint4 v, bool seen, bool& noted) {
  if (!seen) return make_uint4(0, 0, 0, 0);
  const uint32_t a = nonfinite_mask<kF16>(v.x), b = nonfinite_mask<kF16>(v.y);
  const uint32_t c = nonfinite_mask<kF16>(v.z), d = nonfinite_mask<kF16>(v.w);
  noted = noted || (a | b | c | d) != 0;
  return make_uint4(v.x & ~a, v.y & ~b, v.z & ~c, v.w & ~d);
}

// sum + 0 * v of eight bf16 values: zeros, of either sign, unless v holds an infinity or NaN.
__device__ __forceinline__ void add_times_zero(uint32_t (&sum)[4], uint4 v) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[i]) : "r"(x[i]), "r"(0u));
}

// The same for 16 E4M3 codes (NaN is 0x7f or 0xff; there are no infinities).
__device__ __forceinline__ uint4 clean_codes(uint4 v, bool seen, bool& noted) {
  if (!seen) return make_uint4(0, 0, 0, 0);
  const auto nan = [](uint32_t x) { return (((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7; };
  const uint32_t a = nan(v.x), b = nan(v.y), c = nan(v.z), d = nan(v.w);
  noted = noted || (a | b | c | d) != 0;
  return make_uint4(v.x & ~(a * 0xffu), v.y & ~(b * 0xffu), v.z & ~(c * 0xffu), v.w & ~(d * 0xffu));
}

// Tiles of this CTA out of whose V an infinity or NaN was taken.  Tiles are counted over all items; `last` is one past
// the last such tile, and a slot holds the same for the tiles that fall on it.  Entries only
// grow: one that a later tile has overwritten says yes for an earlier one too, which then is looked
// at without need, and nothing has to be cleared between items.
struct NotedTiles {
  static constexpr int kSlots = 64;
  uint32_t last, slot[kSlots];
  __device__ __forceinline__ void clear(int i) {  // by threads 0 .. kSlots
    if (i < kSlots)
      slot[i] = 0;
    else if (i == kSlots)
      last = 0;
  }
  __device__ __forceinline__ void note(uint32_t t) {
    *static_cast<volatile uint32_t*>(&slot[t % kSlots]) = t + 1;  // (warps are less than kSlots tiles apart)
    atomicMax(&last, t + 1);                                      // a slower warp may note the tile before
  }
  // one answer for the warp: another one may be noting a later tile meanwhile
  __device__ __forceinline__ bool any_since(uint32_t t) const volatile { return __any_sync(0xffffffffu, last > t); }
  __device__ __forceinline__ bool at(uint32_t t) const volatile { return __any_sync(0xffffffffu, slot[t % kSlots] > t); }
};

// Element offset of a key's first value of kv head h, and one value of a pool.
__device__ __forceinline__ int64_t value_at(const AttnJob& p, int page, int h, int key, int dim) {
  return page * p.page_stride +
         ((static_cast<int64_t>(h) << p.page_log2) + (key & ((1 << p.page_log2) - 1))) * dim;
}
template <bool kFp8>
__device__ __forceinline__ float pool_value(const void* pool, int64_t at) {
  if constexpr (kFp8) {
    uint32_t x, y;
    e4m3x4_to_f16x2(*(static_cast<const uint8_t*>(pool) + at), x, y);
    return f16lo_to_f32(x);
  } else {
    return bf16_bits_to_f32(*(static_cast<const uint16_t*>(pool) + at));
  }
}

// Whether kValues values of a pool from element `at` on (16-byte aligned) hold an infinity or NaN.
template <bool kFp8, int kValues>
__device__ __forceinline__ bool holds_nonfinite(const void* pool, int64_t at) {
  constexpr int kEl = kFp8 ? 1 : 2;
  const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(pool) + at * kEl);
  bool noted = false;
#pragma unroll 4
  for (int i = 0; i < kValues * kEl / 16; ++i) {
    if constexpr (kFp8)
      clean_codes(v[i], true, noted);
    else
      clean_chunk<false>(v[i], true, noted);
  }
  return noted;
}

__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

// Byte offset of chunk c (16 bytes) of row r in a block of rows, swizzled as the boxes are.
template <typename T>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  const uint32_t o = r * T::kRowB + c * 16;
  return o ^ ((o >> 3) & T::kSwz);
}

// Byte offset of the first block's row r (a multiple of 8) in a unit's K or V, which lies
// there in page pieces of [kSub][1 << piece_log2][kRowB].
template <typename T>
__device__ __forceinline__ uint32_t rows_at(int r, int piece_log2) {
  return r * T::kRowB + ((r >> piece_log2) * (T::kSub - 1) << piece_log2) * T::kRowB;
}

// The page of piece `piece` (1 << piece_log2 keys) of a sequence, or -1 if it holds no
// key of the tile; a page id outside the pool becomes num_pages, a coordinate past the
// tensor map's end, which reads as zeros.
__device__ __forceinline__ int piece_page(const AttnJob& p, const int32_t* table, int piece, int piece_log2,
                                          const RowTile& t) {
  const int k = piece << piece_log2;
  if (k >= t.hi || k + (1 << piece_log2) <= t.lo) return -1;  // holds no key of [lo, hi): not copied
  const int page = __ldg(table + (k >> p.page_log2));
  if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) return page;
  atomicOr(&g_device_error, kErrPage);
  return p.num_pages;
}

// ------------------------------------------------------------------ the split kernel

template <int kDim, bool kFp8, int kRW, int kKW, bool kTree>
__global__ void __launch_bounds__(AttnTile<kDim, kFp8, kRW, kKW>::kThreadsAll, attn_ctas(kDim, kFp8, kRW))
    attn_split_kernel(const AttnJob p, const __grid_constant__ KvMaps maps) {
  using T = AttnTile<kDim, kFp8, kRW, kKW>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  const uint32_t q_at = ring + T::kStages * T::kStageB, join = q_at + T::kQB;
  uint8_t* tail = smem_raw + (join + T::kJoinB - raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(tail);  // [stages]
  uint64_t* empty = full + T::kStages;                 // [stages]
  RangeScratch* scratch = reinterpret_cast<RangeScratch*>(empty + T::kStages);
  float* q_back = reinterpret_cast<float*>(scratch + 1);  // [kRows] undoes the scaling of a row of Q
  NotedTiles* const noted_tiles = reinterpret_cast<NotedTiles*>(q_back + T::kRows);
  static_assert(2 * 6 * sizeof(uint64_t) + sizeof(RangeScratch) + 64 * sizeof(float) + sizeof(NotedTiles) <= 1024, "tail");

  const int warp = static_cast<int>(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < T::kStages; ++i) mbar_init(full + i, 1), mbar_init(empty + i, T::kConsumers);
    fence_mbar_init();
  }
  noted_tiles->clear(threadIdx.x);
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();

  constexpr auto kTiling = tiling_for<kTree>(T::tiling());
  Found f;
  Ranges ranges;
  find_range<T::kThreadsAll>(p, kTiling, gridDim.x, blockIdx.x, &ranges, &f, scratch,
                             reinterpret_cast<longlong2*>(smem_raw + (ring - raw)));
  // (the list lies where the first tiles will: its last reads come before the copies)
  fence_proxy_async_smem();
  __syncthreads();
  if (threadIdx.x == T::kConsumers * 32) p.split[blockIdx.x] = make_int4(0, 0, 0, 0);  // none, until this thread finds one
  if (static_cast<int>(blockIdx.x) >= ranges.grid) return;
  const long long u0 = ranges.start(blockIdx.x), u1 = ranges.start(blockIdx.x + 1);
  Walk w;
  w.b = f.seq, w.item0 = f.before;
  walk_seq(p, w, kTiling);

  bool ran_out = false;  // a wait reached its limit (recorded): no further waits, the roles stay in step
  if (warp == T::kConsumers) {
    // -------------------------------------------------------------- producer
    const int piece_log2 = min(p.page_log2, log2c(T::kKeys));
    constexpr int kMostPieces = T::kKeys / 16;
    const int pieces = T::kKeys >> piece_log2;  // of a unit: at most kMostPieces
    const uint32_t bytes = 2u << piece_log2 << log2c(kDim * T::kEl);
    int st = 0;
    uint32_t round = 0;
    for (long long u = u0; u < u1 && !ran_out;) {
      walk_to(p, w, u, kTiling);
      const Share pc = share_at(w, u, u0, u1, blockIdx.x, kTiling);
      u = pc.end;
      const int n = static_cast<int>(uniform(pc.n)), head = static_cast<int>(uniform(w.h));
      if (n > 0 && !pc.whole && pc.first == w.t.tile0 && lane == 0)
        p.split[blockIdx.x] = split_item(w, holders_of(w, ranges, kTiling).c1);
      const int32_t* table = p.table + static_cast<int64_t>(w.b) * p.max_pages;
      // lane i holds the page of piece i of the unit, looked up a unit ahead
      int page = lane < pieces && n > 0 ? piece_page(p, table, pc.first * pieces + lane, piece_log2, w.t) : -1;
      for (int i = 0; i < n; ++i) {
        const int later = lane < pieces && i + 1 < n
                              ? piece_page(p, table, (pc.first + i + 1) * pieces + lane, piece_log2, w.t) : -1;
        ran_out = round > 0 && !mbar_wait_warp(empty + st, (round - 1) & 1);
        if (ran_out) break;
        const uint32_t bar = smem_addr(full + st);
        const uint32_t all = bytes * __popc(__ballot_sync(0xffffffffu, page >= 0));
        int at[kMostPieces];  // all pieces' pages first, then the copies back to back
#pragma unroll
        for (int j = 0; j < kMostPieces; ++j) at[j] = __shfl_sync(0xffffffffu, page, j);
        if (elect_one()) {
          mbar_arrive_expect_tx_s(bar, all);
#pragma unroll
          for (int j = 0; j < kMostPieces; ++j) {
            if (j >= pieces) break;
            if (at[j] < 0) continue;
            const uint32_t dst = ring + st * T::kStageB + (j << piece_log2) * (kDim * T::kEl);
            const int row = (((pc.first + i) * pieces + j) << piece_log2) & ((1 << p.page_log2) - 1);
            tma_load_5d(dst, &maps.k, 0, row, 0, head, at[j], bar);
            tma_load_5d(dst + T::kTileB, &maps.v, 0, row, 0, head, at[j], bar);
          }
        }
        __syncwarp();
        page = later;
        if (++st == T::kStages) st = 0, ++round;
      }
    }
    // the CTA's shared memory is its own until its last copies have landed, whatever ran out (bounded)
    const uint32_t issued = round * T::kStages + st;
    for (uint32_t i = issued > T::kStages ? issued - T::kStages : 0; i < issued; ++i)
      (void)mbar_wait_warp(full + i % T::kStages, i / T::kStages & 1);
    return;
  }

  // ---------------------------------------------------------------- consumers
  const int rw = warp % kRW, kw = warp / kRW;
  const int g = lane >> 2, t4 = lane & 3;
  constexpr int kNT = T::kSlice / 8;      // key columns of 8
  constexpr int kDT = kDim / 8;           // value columns of 8
  constexpr int kKS = kDim / 16;          // k steps of the first product
  const float log2e = 1.4426950408889634f;
  // ldmatrix addresses: for K lane l gives row l % 8 of chunk l / 8, for V and Q row l % 16
  // of chunk l / 16; chunk c of a row lies at c * 16 bytes, its low bits exchanged by the row's
  const int piece_log2 = min(p.page_log2, log2c(T::kKeys));
  const uint32_t block = T::kRowB << piece_log2;  // bytes from one 128-byte block of a piece to the next
  const uint32_t k_lane = swizzled<T>(lane & 7, lane >> 3), v_lane = swizzled<T>(lane & 15, lane >> 4);
  const uint32_t q_lane = q_at + rw * 16 * 128 + ((lane & 15) * 128 | (((lane >> 4) ^ (lane & 7)) << 4));
  int st = 0;
  uint32_t round = 0;

  for (long long u = u0; u < u1;) {
    walk_to(p, w, u, kTiling);
    const Share pc = share_at(w, u, u0, u1, blockIdx.x, kTiling);
    u = pc.end;
    if (pc.n == 0) continue;

    // this thread's two rows (g and g + 8 of the warp's 16): token, head, position
    int pos[2], tok[2], head[2];
    bool live[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = rw * 16 + g + 8 * i;
      live[i] = r < w.t.rows;
      const int rr = w.t.row0 + min(r, w.t.rows - 1);
      tok[i] = div_by(p.by_group, rr);
      head[i] = w.h * p.group + rr - tok[i] * p.group;
      pos[i] = w.s.len - w.s.n + tok[i];
    }
    // positions over the warp's rows: the smallest and largest
    const int r_lo = w.t.row0 + min(rw * 16, w.t.rows - 1), r_hi = w.t.row0 + min(rw * 16 + 15, w.t.rows - 1);
    const int pos_lo = w.s.len - w.s.n + div_by(p.by_group, r_lo);
    const int pos_hi = w.s.len - w.s.n + div_by(p.by_group, r_hi);
    int all_hi = min(pos_lo + 1, w.s.len);                                        // keys [all_lo, all_hi) seen by every row
    int all_lo = p.window > 0 ? pos_hi - p.window + 1 : 0;
    int any_hi = min(pos_hi + 1, w.s.len);                                        // keys [any_lo, any_hi) seen by some row
    int any_lo = p.window > 0 ? max(pos_lo - p.window + 1, 0) : 0;

    // keys that every row of the item sees, or some row (the tiles between are cleaned)
    const KeyRange kr = key_range<kTree>(p, w);
    if constexpr (kTree) all_hi = kr.all_hi, all_lo = kr.all_lo, any_hi = kr.any_hi, any_lo = kr.any_lo;

    // Q to shared memory, each warp a quarter of the rows, eight lanes a row
    if constexpr (kKW > 1) asm volatile("bar.sync 1, %0;" ::"n"(T::kConsumers * 32) : "memory");  // the last item's Q is read
#pragma unroll
    for (int it = 0; it < T::kRows / (4 * T::kConsumers); ++it) {
      const int r = (kKW > 1 ? warp : rw) * (T::kRows / T::kConsumers) + 4 * it + (lane >> 3);
      const int rr = w.t.row0 + min(r, w.t.rows - 1);
      const int tk = div_by(p.by_group, rr), hd = w.h * p.group + rr - tk * p.group;
      const uint16_t* q = p.q + (w.s.tok0 + tk) * p.q_stride + static_cast<int64_t>(hd) * kDim;
      const bool zero = r >= w.t.rows;
      uint4 v[kDim / 64];
#pragma unroll
      for (int c = 0; c < kDim / 64; ++c)
        v[c] = zero ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(q + 64 * c + 8 * (lane & 7));
      if (p.scale == 0.f) {
#pragma unroll
        for (int c = 0; c < kDim / 64; ++c) v[c] = zero_or_nan(v[c]);
      }
      const uint32_t sign = p.scale < 0.f ? 0x80008000u : 0u;  // a negative scale turns q's sign
      if constexpr (!kFp8) {
#pragma unroll
        for (int c = 0; c < kDim / 64; ++c)
          sts128(q_at + c * T::kRows * 128 + r * 128 + (((lane & 7) ^ (r & 7)) << 4),
                 make_uint4(v[c].x ^ sign, v[c].y ^ sign, v[c].z ^ sign, v[c].w ^ sign));
      } else {
        // scaled into f16's range; the pairs of 16 values in the order in which the codes of a
        // key come out of ldmatrix (pairs 0, 2, 4, 6, then 1, 3, 5, 7)
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < kDim / 64; ++c) {
          const uint32_t x[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[j] << 16)), fabsf(__uint_as_float(x[j] & 0xffff0000u))));
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int e = pow2_rescale_exponent(amax);
        const float up = exp2i(e);
        if ((lane & 7) == 0) q_back[r] = exp2i(-e);
#pragma unroll
        for (int c = 0; c < kDim / 64; ++c) {
          uint32_t x[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[j] ^= sign;
            x[j] = f32x2_to_f16x2(__uint_as_float(x[j] << 16) * up, __uint_as_float(x[j] & 0xffff0000u) * up);
          }
          const uint32_t row = q_at + c * T::kRows * 128 + r * 128 + 8 * (lane & 1);
          const int even = lane & 6;
          sts64(row + ((even ^ (r & 7)) << 4), x[0], x[2]);
          sts64(row + (((even + 1) ^ (r & 7)) << 4), x[1], x[3]);
        }
      }
    }
    if constexpr (kKW > 1)
      asm volatile("bar.sync 1, %0;" ::"n"(T::kConsumers * 32) : "memory");
    else
      __syncwarp();
    const float ks = (kFp8 && p.k_scale) ? __ldg(p.k_scale + w.h) : 1.0f;
    // logits in units of log 2: acc * mul; with a softcap, cap2 * tanh(acc * mul)
    const bool capped = p.softcap > 0.f;
    const float unit = (p.scale == 0.f ? 1.0f : fabsf(p.scale)) * ks * (capped ? 1.0f / p.softcap : log2e);
    float mul[2] = {unit, unit};
    if constexpr (kFp8) mul[0] *= q_back[rw * 16 + g], mul[1] *= q_back[rw * 16 + g + 8];
    const float cap2 = p.softcap * log2e;
    // with a softcap the logits are finished before the maximum is taken
    const float fac[2] = {capped ? 1.0f : fmaxf(mul[0], 1.2e-38f), capped ? 1.0f : fmaxf(mul[1], 1.2e-38f)};

    float acc[kDT][4];
#pragma unroll
    for (int j = 0; j < kDT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY};  // reference of the weights: weight = 2^(s - m)
    float l[2] = {0.f, 0.f};              // this lane's share of the sum of weights

    for (int i = 0; i < pc.n; ++i) {
      ran_out = ran_out || !mbar_wait_warp(full + st, round & 1);
      const int key0 = (pc.first + i) * T::kKeys + kw * T::kSlice;
      if (key0 < any_hi && key0 + T::kSlice > any_lo) {
        const uint32_t kt = ring + st * T::kStageB, vt = kt + T::kTileB;
        // ---- s = q . k
        float s[kNT][4];
#pragma unroll
        for (int j = 0; j < kNT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
        uint32_t at[kNT];
#pragma unroll
        for (int j = 0; j < kNT; ++j) at[j] = kt + rows_at<T>(kw * T::kSlice + 8 * j, piece_log2);
        if constexpr (!kFp8) {
#pragma unroll
          for (int k = 0; k < kKS; k += 2) {
            uint32_t a0[4], a1[4];
            ldsm4(a0, q_lane + (k / 4) * T::kRows * 128 ^ ((k & 2) << 5));
            ldsm4(a1, q_lane + (k / 4) * T::kRows * 128 ^ ((k & 2) << 5 | 32));
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
              uint32_t b[4];
              ldsm4(b, at[j] + (k / 4) * block + (k_lane ^ ((k & 2) << 5)));
              mma_16<false>(s[j], a0, b[0], b[1]);
              mma_16<false>(s[j], a1, b[2], b[3]);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < kKS; k += 4) {
            uint32_t a[4][4];
#pragma unroll
            for (int x = 0; x < 4; ++x) ldsm4(a[x], q_lane + (k / 4) * T::kRows * 128 ^ (x << 5));
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
              uint32_t b[4];
              ldsm4(b, at[j] + (k / 8) * block + (k_lane ^ (T::kRowB == 128 ? (k & 4) << 4 : 0)));
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                uint32_t b0, b1;
                e4m3x4_to_f16x2(b[x], b0, b1);
                mma_16<true>(s[j], a[x], b0, b1);
              }
            }
          }
        }
        // ---- softcap, mask, running maximum
        if (capped) {
          float high = 0.f;
#pragma unroll
          for (int j = 0; j < kNT; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[j][x] *= mul[x >> 1], high = fmaxf(high, fabsf(s[j][x]));
          if (__any_sync(0xffffffffu, high >= kTanhSmall)) {
#pragma unroll
            for (int j = 0; j < kNT; ++j)
#pragma unroll
              for (int x = 0; x < 4; ++x) s[j][x] = cap2 * tanh_any(s[j][x]);
          } else {
#pragma unroll
            for (int j = 0; j < kNT; ++j)
#pragma unroll
              for (int x = 0; x < 4; x += kTree ? 2 : 1) {
                if constexpr (kTree) {
                  const f32x2 y = mul2(pack2(cap2, cap2), tanh_small2(pack2(s[j][x], s[j][x + 1])));
                  s[j][x] = lo2(y), s[j][x + 1] = hi2(y);
                } else {
                  s[j][x] = cap2 * tanh_small(s[j][x]);
                }
              }
          }
        }
        if (kTree && (key0 + T::kSlice > all_hi || key0 < all_lo)) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const TreeRow row = tree_row(p, w.s, tok[y]);
#pragma unroll
            for (int j0 = 0; j0 < kNT; j0 += 4) {
              const uint32_t seen = row.bits(key0 + 8 * j0) >> (2 * t4);
#pragma unroll
              for (int j = j0; j < kNT && j < j0 + 4; ++j)
#pragma unroll
                for (int x = 0; x < 2; ++x) s[j][2 * y + x] = seen >> (8 * (j - j0) + x) & 1 ? s[j][2 * y + x] : -INFINITY;
            }
          }
        }
        if (!kTree && (key0 + T::kSlice > all_hi || key0 < all_lo)) {
#pragma unroll
          for (int j = 0; j < kNT; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = key0 + 8 * j + 2 * t4 + (x & 1), ps = pos[x >> 1];
              const bool sees = key <= ps && key < w.s.len && (p.window <= 0 || key > ps - p.window);
              s[j][x] = sees ? s[j][x] : -INFINITY;
            }
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < kNT; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) top[x >> 1] = fmaxf(top[x >> 1], s[j][x]);
        float alpha[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
          top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
          const float next = fmaxf(m[x], top[x] * fac[x] - (kFp8 ? 15.0f : 0.0f));
          // a row that has seen nothing keeps -inf as its reference and 0 as its sum
          alpha[x] = next == -INFINITY ? 1.0f : exp2_approx(m[x] - next);
          m[x] = next;
        }
        const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
        if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
          l[0] *= alpha[0], l[1] *= alpha[1];
#pragma unroll
          for (int j = 0; j < kDT; ++j) {
            acc[j][0] *= alpha[0], acc[j][1] *= alpha[0];
            acc[j][2] *= alpha[1], acc[j][3] *= alpha[1];
          }
        }
#pragma unroll
        for (int j = 0; j < kNT; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            s[j][x] = exp2_approx(fmaf(s[j][x], fac[x >> 1], -ref[x >> 1]));
            l[x >> 1] += s[j][x];
          }
        // ---- out += weights . v, with V cleaned where some row of the item does not see all of
        // the slice: keys that no row sees become zeros (0 * inf is NaN), infinities and NaN
        // are taken out and noted
        if (partly_seen(kr, key0, T::kSlice)) {
          constexpr int kChunks = kDim * T::kEl / 16;
          bool noted = false;
          for (int i = lane; i < T::kSlice * kChunks; i += 32) {
            const int r = kw * T::kSlice + i / kChunks, c = i % kChunks, key = key0 + i / kChunks;
            const uint32_t o = (r & 15) * T::kRowB + (c % (T::kRowB / 16)) * 16;
            const uint32_t a = vt + rows_at<T>(r & ~15, piece_log2) + c / (T::kRowB / 16) * block + (o ^ ((o >> 3) & T::kSwz));
            const bool seen = key >= kr.any_lo && key < kr.any_hi;
            if constexpr (kFp8)
              sts128(a, clean_codes(lds128(a), seen, noted));
            else
              sts128(a, clean_chunk<false>(lds128(a), seen, noted));
          }
          if (noted) noted_tiles->note(round * T::kStages + st);
          fence_proxy_async_smem();  // the stage's next copy comes after these writes
          __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < T::kSlice / 16; ++k) {
          uint32_t a[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float lo = s[2 * k + (x >> 1)][2 * (x & 1)], hi = s[2 * k + (x >> 1)][2 * (x & 1) + 1];
            a[x] = kFp8 ? f32x2_to_f16x2(lo, hi) : f32x2_to_bf16x2(lo, hi);
          }
          [[maybe_unused]] uint32_t r[4];
          const uint32_t rows = vt + rows_at<T>(kw * T::kSlice + 16 * k, piece_log2);
#pragma unroll
          for (int c = 0; c < kDT / 2; ++c) {
            // b: two columns of 8 values each, 16 keys (E4M3: one 16-value chunk)
            uint32_t b[4];
            if constexpr (!kFp8) {
              ldsm4t(b, rows + (c / 4) * block + (v_lane ^ ((c & 3) << 5)));
            } else {
              // matrices: (keys 0-7, chunk c), (keys 8-15, chunk c), then chunk c + 1; a word
              // holds two keys of two adjacent values
              static_assert(kDT % 4 == 0, "chunks come in pairs");
              if (c % 2 == 0) ldsm4t(r, rows + (T::kRowB == 128 ? c / 8 : 0) * block + (v_lane ^ ((c & 6) << 4)));
              const uint32_t w0 = __byte_perm(r[c % 2 ? 2 : 0], 0, 0x3120), w1 = __byte_perm(r[c % 2 ? 3 : 1], 0, 0x3120);
              e4m3x4_to_f16x2(w0, b[0], b[2]);
              e4m3x4_to_f16x2(w1, b[1], b[3]);
            }
            mma_16<kFp8>(acc[2 * c], a, b[0], b[1]);
            mma_16<kFp8>(acc[2 * c + 1], a, b[2], b[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + st);
      if (++st == T::kStages) st = 0, ++round;
    }

    // ---- infinities and NaN that were taken out of V, to the rows that see them
    // (warps that share a slice may each have found it clean already: the note tells)
    if constexpr (kRW > 1) asm volatile("bar.sync 1, %0;" ::"n"(T::kConsumers * 32) : "memory");
    const volatile NotedTiles* const notes = noted_tiles;
    const uint32_t unit0 = round * T::kStages + st - pc.n;  // this item's first unit
    if (notes->any_since(unit0)) {
      for (int i = 0; i < pc.n; ++i) {
        const int key0 = (pc.first + i) * T::kKeys + kw * T::kSlice;
        if (!notes->at(unit0 + i) || !partly_seen(kr, key0, T::kSlice)) continue;
        // each lane looks at one key, then all of them at those that hold any
        const int hi = min(key0 + T::kSlice, kr.any_hi);
#pragma unroll 1
        for (int k0 = max(key0, kr.any_lo); k0 < hi; k0 += 32) {
          int64_t mine = 0;
          bool holds = false;
          if (k0 + lane < hi) {
            const int page = __ldg(p.table + static_cast<int64_t>(w.b) * p.max_pages + ((k0 + lane) >> p.page_log2));
            mine = value_at(p, page, w.h, k0 + lane, kDim);
            holds = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages) &&
                    holds_nonfinite<kFp8, kDim>(p.v_pool, mine);
          }
#pragma unroll 1
          for (unsigned left = __ballot_sync(0xffffffffu, holds); left; left &= left - 1) {
            const int who = __ffs(left) - 1, key = k0 + who;
            const int64_t at = __shfl_sync(0xffffffffu, mine, who);
            [[maybe_unused]] bool sees[2];
            if constexpr (kTree) {
#pragma unroll
              for (int y = 0; y < 2; ++y) sees[y] = tree_row(p, w.s, tok[y]).sees(key);
            }
#pragma unroll
            for (int j = 0; j < kDT; ++j)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                // the column of acc[j][x] (E4M3: see the store below)
                const int col = kFp8 ? 16 * (j / 2) + 4 * t4 + 2 * x + (j & 1) : 8 * j + 2 * t4 + x;
                const float v = pool_value<kFp8>(p.v_pool, at + col);
                if (isfinite(v)) continue;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  if constexpr (kTree) {
                    if (sees[y]) acc[j][2 * y + x] += v;
                  } else {
                    if (key <= pos[y] && key < w.s.len && (p.window <= 0 || key > pos[y] - p.window)) acc[j][2 * y + x] += v;
                  }
                }
              }
          }
        }
      }
    }

    // ---- join the key slices of this CTA
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    }
    if constexpr (kKW > 1) {
      float* buf = reinterpret_cast<float*>(smem_raw + (join - raw));
      float4* ml = reinterpret_cast<float4*>(buf + T::kJoinB / 4) - T::kConsumers * 32;  // at the end of the buffer
      ml[warp * 32 + lane] = make_float4(m[0], m[1], l[0], l[1]);
      asm volatile("bar.sync 1, %0;" ::"n"(T::kConsumers * 32) : "memory");
      // one reference and sum for all slices; every warp scales its sums to it
      float f[2];
      float4 o[kKW];
#pragma unroll
      for (int i = 0; i < kKW; ++i) o[i] = ml[(i * kRW + rw) * 32 + lane];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float next = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < kKW; ++i) next = fmaxf(next, x ? o[i].y : o[i].x);
#pragma unroll
        for (int i = 0; i < kKW; ++i)
          sum += (x ? o[i].w : o[i].z) * (next == -INFINITY ? 1.0f : exp2_approx((x ? o[i].y : o[i].x) - next));
        f[x] = next == -INFINITY ? 1.0f : exp2_approx(m[x] - next);
        m[x] = next, l[x] = sum;
      }
#pragma unroll
      for (int j = 0; j < kDT; ++j) acc[j][0] *= f[0], acc[j][1] *= f[0], acc[j][2] *= f[1], acc[j][3] *= f[1];
      // each slice's warp ends with the columns [kw, kw + 1) * kDT / kKW of all slices: in
      // round r it hands slice kw + r that slice's columns
      constexpr int kPart = kDT / kKW;
#pragma unroll 1
      for (int r = 1; r < kKW; ++r) {
        const int dest = (kw + r) % kKW;
        float4* give = reinterpret_cast<float4*>(buf) + (dest * kRW + rw) * 32 * kPart + lane;
#pragma unroll
        for (int q = 0; q < kKW; ++q)
          if (q == dest) {
#pragma unroll
            for (int j = 0; j < kPart; ++j)
              give[j * 32] = make_float4(acc[q * kPart + j][0], acc[q * kPart + j][1], acc[q * kPart + j][2], acc[q * kPart + j][3]);
          }
        asm volatile("bar.sync 1, %0;" ::"n"(T::kConsumers * 32) : "memory");
        const float4* take = reinterpret_cast<const float4*>(buf) + (kw * kRW + rw) * 32 * kPart + lane;
#pragma unroll
        for (int q = 0; q < kKW; ++q)
          if (q == kw) {
#pragma unroll
            for (int j = 0; j < kPart; ++j) {
              const float4 v = take[j * 32];
              acc[q * kPart + j][0] += v.x, acc[q * kPart + j][1] += v.y;
              acc[q * kPart + j][2] += v.z, acc[q * kPart + j][3] += v.w;
            }
          }
        asm volatile("bar.sync 1, %0;" ::"n"(T::kConsumers * 32) : "memory");
      }
    }
    // ---- write: the finished rows, or this share of them; each key slice's warp its columns
    constexpr int kOut = kDT / kKW;
    float vs = 1.0f;
    if constexpr (kFp8) vs = p.v_scale ? __ldg(p.v_scale + w.h) : 1.0f;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (!live[x]) continue;
      const int64_t row = w.s.tok0 + tok[x];
      const int r = rw * 16 + g + 8 * x;
      const float inv = l[x] == 0.f ? 0.f : vs / l[x];
      uint16_t* o = p.out + row * p.out_stride + static_cast<int64_t>(head[x]) * kDim;
      float* part = p.part + (static_cast<int64_t>(pc.slot) * T::kRows + r) * kDim;
#pragma unroll
      for (int q = 0; q < kKW; ++q)
        if (q == kw) {
#pragma unroll
          for (int j = q * kOut; j < (q + 1) * kOut; j += 2) {
            const float v0 = acc[j][2 * x], v1 = acc[j][2 * x + 1], v2 = acc[j + 1][2 * x], v3 = acc[j + 1][2 * x + 1];
            if constexpr (!kFp8) {
              if (pc.whole) {
                *reinterpret_cast<uint32_t*>(o + 8 * j + 2 * t4) = f32x2_to_bf16x2(v0 * inv, v1 * inv);
                *reinterpret_cast<uint32_t*>(o + 8 * j + 8 + 2 * t4) = f32x2_to_bf16x2(v2 * inv, v3 * inv);
              } else {
                *reinterpret_cast<float2*>(part + 8 * j + 2 * t4) = make_float2(v0, v1);
                *reinterpret_cast<float2*>(part + 8 * j + 8 + 2 * t4) = make_float2(v2, v3);
              }
            } else {  // (columns j and j + 1 hold alternate values)
              if (pc.whole)
                *reinterpret_cast<uint2*>(o + 8 * j + 4 * t4) =
                    make_uint2(f32x2_to_bf16x2(v0 * inv, v2 * inv), f32x2_to_bf16x2(v1 * inv, v3 * inv));
              else
                *reinterpret_cast<float4*>(part + 8 * j + 4 * t4) = make_float4(v0, v2, v1, v3);
            }
          }
        }
      if (kw == 0 && t4 == 0) {
        if (!pc.whole) {
          float* ml = p.part + static_cast<int64_t>(2) * gridDim.x * T::kRows * kDim;
          *reinterpret_cast<float2*>(ml + (static_cast<int64_t>(pc.slot) * T::kRows + r) * 2) = make_float2(m[x], l[x]);
        } else if (p.lse) {
          p.lse[row * p.n_heads + head[x]] = l[x] == 0.f ? -INFINITY : (m[x] + log2f(l[x])) * 0.6931471805599453f;
        }
      }
    }
  }
}

// ------------------------------------------------------------------ the join

constexpr int kJoinWarps = 8, kJoinThreads = 32 * kJoinWarps, kJoinGrid = 4 * kAttnGrid;
constexpr int kJoinSlices = 4;  // warps on a row's shares, where rows are few

// Joins the shares of the split kernel's split items.  Every block compacts the list of split
// items, and their rows are dealt to the grid: a warp a row where that keeps the grid busy (48
// sequences of 1,000 keys with 64 rows of 64 values: 43 us with four warps a row, 28 with one),
// else kJoinSlices.  Bound by latency: the list,
// then a row's shares, kBatch loads a lane in flight (128 registers; with 64 the loads go in turn, and one
// sequence of 32,000 keys, 76 shares, 8 rows of 128 values, takes 26.5 us instead of 22.5).
// Eight warps a row: 21.3 us there, but verify blocks of 30 rows of 256 values 17.1 instead of
// 15.9; two (before that step): 31.9 against 26.1; a block for every range boundary, most of
// them idle, and a warp a row: 38.4.  Joined by the last CTA to arrive, without this grid,
// verify blocks take 23 us, as one CTA then reads all shares of 30 rows.
template <int kDim>
__global__ void __launch_bounds__(kJoinThreads, 2) attn_join_kernel(const AttnJob p, int split_grid, int tile_rows) {
  __shared__ int warp_sum[(2 * kAttnGrid + kJoinThreads - 1) / kJoinThreads * kJoinWarps];
  __shared__ int4 list[kAttnGrid * 2];
  __shared__ float sums[kJoinWarps][kDim];
  __shared__ float2 refs[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kSpan = (2 * kAttnGrid + kJoinThreads - 1) / kJoinThreads;
  int4 mine[kSpan];
  unsigned all[kSpan];
#pragma unroll
  for (int b = 0; b < kSpan; ++b) {
    const int c = b * kJoinThreads + threadIdx.x;
    mine[b] = c < split_grid ? __ldcg(p.split + c) : make_int4(0, 0, 0, 0);
  }
#pragma unroll
  for (int b = 0; b < kSpan; ++b) {
    all[b] = __ballot_sync(0xffffffffu, mine[b].x != 0);
    if (lane == 0) warp_sum[b * kJoinWarps + warp] = __popc(all[b]);
  }
  __syncthreads();
  int items = 0;
#pragma unroll
  for (int b = 0; b < kSpan; ++b) {
    int at = __popc(all[b] & ((1u << lane) - 1));
#pragma unroll
    for (int x = 0; x < kJoinWarps; ++x) {
      if (x == warp) at += items;
      items += warp_sum[b * kJoinWarps + x];
    }
    if (mine[b].x != 0) list[at] = make_int4(mine[b].x | (b * kJoinThreads + threadIdx.x) << 16, mine[b].y, mine[b].z, mine[b].w);
  }
  __syncthreads();
  const float* ml = p.part + static_cast<int64_t>(2) * split_grid * tile_rows * kDim;
  // kBatch of a row's shares are in flight in each of the warps that they are dealt to (one item
  // of 32,000 keys over the whole grid has 76 shares)
  constexpr int kPer = kDim / 32, kBatch = kDim == 256 ? 4 : 8;
  const int slices = items * tile_rows >= kJoinGrid * kJoinWarps ? 1 : kJoinSlices, per = kJoinWarps / slices;
  const int slice = warp % slices, sub = warp / slices;
  for (int x = blockIdx.x; x < items * (tile_rows / per); x += gridDim.x) {
    const int r0 = x / items * per;
    const int4 it = list[x - x / items * items];
    const int c0 = it.x >> 16, c1 = it.x & 0x1ff, rows = it.x >> 9 & 0x7f;
    if (r0 >= rows) continue;
    const int r = min(r0 + sub, rows - 1);
    float m = -INFINITY, l = 0.f, acc[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) acc[j] = 0.f;
    for (int i0 = c0 + slice; i0 <= c1; i0 += slices * kBatch) {
      float2 v[kBatch], x[kBatch][kPer / 2];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * slices;
        v[k] = make_float2(-INFINITY, 0.f);
        if (i > c1) continue;
        const int64_t row = static_cast<int64_t>(2 * i + (i == c0 ? 1 : 0)) * tile_rows + r;
        v[k] = *reinterpret_cast<const float2*>(ml + row * 2);
        const float2* o = reinterpret_cast<const float2*>(p.part + row * kDim + lane * kPer);
#pragma unroll
        for (int j = 0; j < kPer / 2; ++j) x[k][j] = o[j];
      }
      float next = m;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) next = fmaxf(next, v[k].x);
      const float a0 = next == -INFINITY ? 1.0f : exp2_approx(m - next);
      l *= a0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) acc[j] *= a0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (i0 + k * slices > c1) break;
        const float a = next == -INFINITY ? 1.0f : exp2_approx(v[k].x - next);
        l += a * v[k].y;
#pragma unroll
        for (int j = 0; j < kPer; j += 2) acc[j] += a * x[k][j / 2].x, acc[j + 1] += a * x[k][j / 2].y;
      }
      m = next;
    }
    if (slices > 1) {  // the slices in their order
#pragma unroll
      for (int j = 0; j < kPer; j += 2)
        *reinterpret_cast<float2*>(&sums[warp][lane * kPer + j]) = make_float2(acc[j], acc[j + 1]);
      if (lane == 0) refs[warp] = make_float2(m, l);
      __syncthreads();
      if (slice == 0) {
#pragma unroll
        for (int k = 1; k < kJoinSlices; ++k) m = fmaxf(m, refs[warp + k].x);
        l = 0.f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) acc[j] = 0.f;
#pragma unroll
        for (int k = 0; k < kJoinSlices; ++k) {
          const float a = m == -INFINITY ? 1.0f : exp2_approx(refs[warp + k].x - m);
          l += a * refs[warp + k].y;
#pragma unroll
          for (int j = 0; j < kPer; ++j) acc[j] += a * sums[warp + k][lane * kPer + j];
        }
      }
      __syncthreads();
    }
    if (slice == 0 && r0 + sub < rows) {
      const int rr = it.z + r, tok = div_by(p.by_group, rr), head = it.y * p.group + rr - tok * p.group;
      const int64_t row = it.w + tok;
      const float inv = l == 0.f ? 0.f : (p.v_scale ? __ldg(p.v_scale + it.y) : 1.0f) / l;
      uint32_t* o = reinterpret_cast<uint32_t*>(p.out + row * p.out_stride + static_cast<int64_t>(head) * kDim) + lane * (kPer / 2);
#pragma unroll
      for (int j = 0; j < kPer; j += 2) o[j / 2] = f32x2_to_bf16x2(acc[j] * inv, acc[j + 1] * inv);
      if (p.lse && lane == 0) p.lse[row * p.n_heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
  }
}

// ------------------------------------------------------------------ launch

// Which kernel and tile serve up to `rows` packed rows per sequence and kv head, in `items`
// pairs of those.
// Rows above 64 go to the tcgen05 kernel (attention_chunk.cuh): 8 sequences of 8,000 keys (128 values,
// bf16), 124 rows: 41 us there, 54 with tiles of 64 rows here.  Heads of 256 values go there above
// 32 rows too, where the batch alone fills the chip: 64 ragged sequences of up to 4,000 keys and 4 kv
// heads, 40 rows, 47 us there and 57 here, 16 of 8,000 keys with 64 rows 107 and 136 (E4M3 106 and 152); but one of
// 32,000 keys 68 and 48, two of 2,000 31 and 19.  With 128 values the ragged batch takes
// 39 us there and 31 here, 48 sequences of 1,000 keys 41 and 43, and only equal lengths gain (16 of
// 8,000 keys 67 and 76, 32 of 500 keys 16 and 24); 64 values likewise (32 and 20, 31 and 28).
// Up to 32 rows this kernel is ahead in every batch measured.
// A tile of 16 rows leaves four key slices to four warps, 32 rows two, 64 rows share one: the smallest
// that holds the rows.  16 sequences of 8,000 keys, 8 rows, 128 values: 51.7, 56.1 and 69.4 us
// with tiles of 16, 32 and 64 rows (E4M3 35.7, 44.4, 92.6); 32 rows: 62.6 and 72.9 us with the latter two.
struct AttnShape {
  int rw, kw, tile_rows, box_keys;
  bool chunk;
  int maps;  // which of a cache's pairs of tensor maps
  bool pair = false;        // two CTAs an SM (attention_chunk.cuh)
  bool whole_rows = !chunk;  // boxes of whole rows, or of 128 bytes of them
};
constexpr int kMapPairs = 4;
inline AttnShape attn_shape(int dim, bool fp8, int64_t rows, int64_t items) {
  if (rows > 64 || (dim == 256 && rows > 32 && items >= 48)) return {0, 0, dim == 256 ? 128 : 256, dim == 256 ? 64 : 128, true, 3};
  const int rw = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
  const int kw = 4 / rw;
  return {rw, kw, 16 * rw, attn_slice(dim, fp8, kw) * kw, false, rw / 2};
}

// The same for a tree_attention call, in `items` pairs of a sequence and a kv head.  The join of its tcgen05 kernel is a
// second grid's (attention_chunk.cuh), which makes that kernel the faster one from fewer rows on, and up to 128 rows of
// heads of 64 and 128 values it runs as two CTAs an SM.
// That kernel and the split kernel, us (1, 2, 4, 8 sequences of 1,000 to 2,000 keys are 8, 16, 32, 64 items):
// 128 values, 60 rows: one sequence of 1,000 keys 12.8 and 14.5 (E4M3 14.3 and 13.9), of 32,000 39 and 45 (37 and 43), two
// 16 and 20 (17.5 and 18.2), four 17 and 25 (20 and 24), 16 of 8,000 96 and 130 (95 and 148), 64 ragged ones 53 and 88
// (49 and 75).  30 rows: one 12.1 and 11.7, two 14.5 and 13.5, four 16.1 and 17.4, eight 19 and 22, 16 of 8,000 93 and 100,
// 64 ragged ones 45 and 54; E4M3 12.6 and 12.0, 18.7 and 18.4, 22 and 23, 95 and 91, 50 and 49.  16 rows: 12 and 11,
// 93 and 93, 48 and 46 (E4M3 13 and 12, 95 and 61, 41 and 28).
// 64 values, 60 rows: one 11.8 and 11.6, of 32,000 keys 26 and 24 (E4M3 29 and 27), two 13.8 and 14.7 (15.1 and 15.6), four 15
// and 17, 64 ragged ones 33 and 38 (38 and 43).  30 rows: eight 15.9 and 16.4, 16 of 8,000 67 and 60, 64 ragged ones 36 and 32.
// 256 values (one CTA an SM), 60 rows: one 15.5 and 16.8 (E4M3 18.0 and 16.8), two 17 and 26 (21 and 26), 16 of 8,000 175 and 243
// (176 and 272).  30 rows: one 12.7 and 14.6, four 20 and 25, 16 of 8,000 171 and 183; E4M3 15.6 and 14.4, four 26.0 and 25.3, eight
// 33.2 and 33.0, 16 of 8,000 175 and 193, 64 ragged ones 82 and 101.  16 rows: four 20 and 18, 16 of 8,000 170 and 164 (172 and 109).
inline AttnShape tree_shape(int dim, bool fp8, int64_t rows, int64_t items, int page_size) {
  if (dim == 256) {
    if (rows > 32 || (rows > 16 && (!fp8 || items >= 64))) return {0, 0, 128, 64, true, 3};
  } else if (rows <= 128 && (rows > 64 || (rows > 32 && (dim == 128 || items >= 16)) ||
                             (rows > 16 && dim == 128 && !fp8 && items >= 32))) {
    // tiles of 64 keys: of pages up to that size by the boxes of the larger tiles, of larger pages by the boxes of 64
    // whole rows that the split kernel has (which lie in a tile as the products read it)
    static_assert(attn_slice(128, false, 4) * 4 == 64 && attn_slice(128, true, 2) * 2 == 64 &&
                  attn_slice(64, false, 2) * 2 == 64 && attn_slice(64, true, 2) * 2 == 64, "boxes");
    if (page_size <= 64) return {0, 0, 128, 128, true, 3, true, false};
    return {0, 0, 128, 64, true, dim == 128 && !fp8 ? 0 : 1, true, true};
  }
  return attn_shape(dim, fp8, rows, items);
}

// Checks of an attention call's sizes.
inline bool attn_rows_ok(int n_tokens, int n_seqs, int max_new, int n_heads, int n_kv_heads, int head_dim) {
  if (n_tokens < 0 || n_seqs < 0 || max_new < 0 || n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads) return false;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return false;
  // positions and packed rows of a sequence are counted in 32 bits
  return n_tokens < (1 << 30) && static_cast<int64_t>(n_tokens) * (n_heads / n_kv_heads) < (int64_t{1} << 31) - 1024;
}
inline bool attn_sizes_ok(int n_tokens, int n_seqs, int max_new, int n_heads, int n_kv_heads, int head_dim,
                          int max_pages, int page_size) {
  // key positions are counted in 32 bits
  return attn_rows_ok(n_tokens, n_seqs, max_new, n_heads, n_kv_heads, head_dim) && (max_pages >= 1 || n_seqs == 0) &&
         static_cast<int64_t>(max_pages) * page_size < (int64_t{1} << 30);
}

inline int64_t packed_rows(int n_tokens, int max_new, int n_heads, int n_kv_heads) {
  return static_cast<int64_t>(n_tokens < max_new ? n_tokens : max_new) * (n_heads / n_kv_heads);
}

inline int attn_window(int window) { return window < (1 << 30) ? window : 0; }  // (no sequence is that long: all keys)

template <int kDim>
nvfp4_status launch_attn_join(const AttnJob& p, int tile_rows, int keys, int grid, cudaStream_t stream) {
  // one unit an item: nothing can be split
  if ((static_cast<int64_t>(p.max_pages) << p.page_log2) > keys &&
      launch_pdl(attn_join_kernel<kDim>, dim3(kJoinGrid), dim3(kJoinThreads), 0, stream, p, grid, tile_rows) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  return launched();
}

template <int kDim, bool kFp8, int kRW, int kKW, bool kTree>
nvfp4_status launch_attn_split(const AttnJob& p, const KvMaps& maps, cudaStream_t stream) {
  using T = AttnTile<kDim, kFp8, kRW, kKW>;
  if (set_smem(attn_split_kernel<kDim, kFp8, kRW, kKW, kTree>, T::kSmem) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (launch_pdl(attn_split_kernel<kDim, kFp8, kRW, kKW, kTree>, dim3(kAttnGrid * T::kCtas), dim3(T::kThreadsAll),
                 T::kSmem, stream, p, maps) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  return launch_attn_join<kDim>(p, T::kRows, T::kKeys, kAttnGrid * T::kCtas, stream);
}

// The split and join grids for heads of kDim values (attention_d*.cu, attention_tree_d*.cu).
template <int kDim, bool kTree>
nvfp4_status dispatch_attention(const AttnJob& p, const KvMaps& maps, bool fp8, const AttnShape& s,
                                cudaStream_t stream);

}  // namespace nvfp4
