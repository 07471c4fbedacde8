// Attention over a paged cache, many rows at a time: prefill chunks and whole
// prompts (paged_attention), on tcgen05 tensor cores with accumulators in TMEM.
//
// The same mathematics, packed rows, units and ranges as the split kernel
// (attention.cuh), with tiles of 128 rows per softmax warpgroup (two of them for
// heads of 64 and 128 values, one for 256) by kKeys keys.
//
// Roles of a CTA (one per SM).  Warp 0 copies K and V tiles by TMA into rings;
// one thread of warp 1 issues every MMA and commits it to mbarriers; two or
// four warps make tiles fit for the tensor cores (below); each softmax warpgroup owns
// 128 rows, a thread a row, so maxima and sums need no exchange.  Per tile: S = Q K^T
// into TMEM; the row's thread reads S, takes weights 2^(s - m), writes them back as
// 16-bit P over S, in two halves; O += P V with P read from TMEM, started on the first half.
// With two row groups the tensor cores run one group's products while the other group is in its
// softmax; with one (256 values: O takes half of TMEM) S is double-buffered and the next
// Q K^T runs meanwhile.  Softcaps and masks rewrite S in TMEM first, so that the common path
// has the registers to hold a whole row of S.
//
// The reference m of a row's weights follows its maximum lazily: only when a new
// maximum exceeds it by 2^8 are the row's sums scaled down, so O rarely leaves the
// tensor cores' hands; weights stay below 2^8 (bf16 holds them as exactly as those below
// 1; f16 weights, for E4M3 caches, are offset by 2^7 and stay below 2^15).
//
// Fit tiles.  For an E4M3 cache the tiles are converted to f16 (exact).  For both
// kinds of cache V is cleaned in tiles that some row does not wholly see: keys outside
// every row's reach become zeros (the pool may hold anything there, and 0 * inf is
// NaN), and an infinity or NaN in a key that only some rows see is taken out of the
// product and noted; the rows that see it add it at the end from the pool itself.
//
// What bounds it.  The last 2,048 tokens over 32,768 keys (32 heads on 8 kv heads of 128 bf16
// values, 1.07 PFLOP) take 695 us, 1.53 PFLOP/s or 80% of cuBLAS's burst rate (768 us under the power cap in a
// long loop, 81% of its sustained one): the softmax of a tile, 128 exponentials a thread, is as
// long as its products.  Short of that, items: a prompt of 4,096 tokens is 512 of them over 152
// CTAs, each with Q to fetch, a first S to wait for and O to write (131 us, 55%; its units alone would take
// 93 at that long chunk's price of one, so that an item's start and end are about 10 us).  Heads of 64 values halve the
// products of a tile but not its softmax.  Heads of 256 values are bound by L2: every CTA reads its own tiles.
#pragma once

#include "attention.cuh"

namespace nvfp4 {

// A ring of stages: the place of tile t, the phase in which it is filled, and the phase in which
// the tile that was there before it is released.
template <int kN>
struct Ring {
  static constexpr int kStages = kN, kLog2 = log2c(kN);
  static __device__ __forceinline__ uint32_t at(uint32_t t) { return t & (kN - 1); }
  static __device__ __forceinline__ uint32_t phase(uint32_t t) { return (t >> kLog2) & 1; }
  static __device__ __forceinline__ bool reused(uint32_t t) { return t >= kN; }
  static __device__ __forceinline__ uint32_t before(uint32_t t) { return ((t >> kLog2) - 1) & 1; }
};

template <int kDim, bool kFp8>
struct ChunkTile {
  static constexpr int kGroups = kDim == 256 ? 1 : 2;      // softmax warpgroups of 128 rows
  static constexpr int kRows = 128 * kGroups;
  static constexpr int kKeys = kDim == 256 ? 64 : 128;
  static constexpr int kSBuf = kDim == 256 ? 2 : 1;        // S buffers per group
  // An item counted as its units alone: a prompt of 4,096 tokens 166 us, with four more 153 (at that
  // step; five more add 2 to 5% to the shorter prompts, two more make it 168).  Boundaries that move up to four
  // units instead of one: 512 tokens in a window of 1,024 keys of 256 values 34.6 us against 35.9, but
  // E4M3 tiles of 128 values, whose units are slow, balance better with one (2,048 tokens 50.8 against 56.7).
  // Ranges of kLeast units or a little less where there are few: 31 tokens over 2,000 keys 25.7 us against 32.8, 33.6 against 46.9 for 256 values.
  static constexpr int kOver = 4, kSnap = kFp8 && kDim == 128 ? 1 : 4, kLeast = kDim == 256 ? 8 : 4;  // in units (Tiling)
  static constexpr __host__ __device__ Tiling tiling() { return {kRows, kKeys, kOver, kSnap, kLeast}; }
  // warps that make tiles fit: two beside the copies and the products, or (E4M3 and 128 values:
  // 256 conversions a row and tile; 830 us with two warps, 705 with four, for 2,048 tokens over
  // 32,768 keys) a warpgroup of their own; the softmax warpgroups follow
  static constexpr bool kFitGroup = kFp8 && kDim == 128;
  static constexpr int kFit0 = kFitGroup ? 4 : 2, kFits = kFitGroup ? 4 : 2, kSoft0 = kFit0 + kFits;
  static constexpr int kThreadsAll = 32 * kSoft0 + 128 * kGroups;
  static constexpr int kEl = kFp8 ? 1 : 2;
  // boxes of the pool (as AttnTile names them, for tile_offset)
  static constexpr int kRowB = kDim * kEl < 128 ? kDim * kEl : 128;
  static constexpr int kSub = kDim * kEl / kRowB;
  static constexpr uint32_t kSwz = kRowB == 128 ? 0x70 : 0x30;
  static constexpr int kSubB = kKeys * kRowB;
  static constexpr int kRawB = kSubB * kSub;               // a K or V tile as it is in the pool
  static constexpr int kTileB = kKeys * kDim * 2;          // a 16-bit tile: [kDim / 64][kKeys][128 bytes]
  static constexpr int kQB = 128 * kDim * 2;               // a group's Q: [kDim / 64][128][128 bytes]
  // stages of the rings (K and V as the products read them, E4M3 tiles as they are copied):
  // powers of two, as many as fit.  E4M3 heads of 64 values: 2,048 tokens 34.2 us against 41.0 with one
  // stage of K and two of V; four stages of copies against two: 2% for 1,500-token pieces.  128 values:
  // 2,048 tokens over 32,768 keys 705 us with two stages of K and two of copies, 1,117 with one and four;
  // 256 values, whose row group waits for copies more than for K, 2,538 and 2,403.
  using KRing = Ring<kDim == 64 ? 4 : (kFp8 && kDim == 256 ? 1 : 2)>;
  using VRing = Ring<kDim == 64 ? 4 : 2>;
  using RawRing = Ring<kDim == 128 ? 2 : 4>;
  static constexpr int kKAt = kGroups * kQB, kVAt = kKAt + KRing::kStages * kTileB;
  static constexpr int kRaw = kVAt + VRing::kStages * kTileB;
  static constexpr int kBars = kRaw + (kFp8 ? RawRing::kStages * kRawB : 0);
  static constexpr size_t kSmem = 1024 + kBars + 1024;
  // TMEM columns: O of each group, then the S buffers
  static constexpr int kSCol = kGroups * kDim;
  static_assert(kSCol + kGroups * kSBuf * kKeys <= 512, "TMEM");
  static_assert(kSmem <= kMaxSmem, "shared memory");
};

// ------------------------------------------------------------------ tcgen05

// Shared-memory matrix descriptor, 128-byte swizzle: start, leading and stride byte
// offsets in units of 16 bytes, version 1.  K-major: rows of 128 bytes, `stride`
// between groups of eight rows.  MN-major: `lead` between blocks of 64 values,
// `stride` between groups of eight k rows.
__device__ __forceinline__ uint64_t umma_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fff) | static_cast<uint64_t>((lead >> 4) & 0x3fff) << 16 |
         static_cast<uint64_t>((stride >> 4) & 0x3fff) << 32 | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: fp32 accumulator, A and B f16 (0) or bf16 (1), B MN-major or
// K-major, N and M.
__device__ __forceinline__ constexpr uint32_t umma_idesc(bool bf16, bool b_mn, int n, int m) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n / 8) << 17) | (static_cast<uint32_t>(m / 16) << 24);
}

constexpr uint32_t kNegateA = 1u << 13;

__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Loaded values are used only after the wait: ties them to this place in the program.
template <int kN>
__device__ __forceinline__ void tmem_loaded(float (&r)[kN]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < kN; ++i) asm volatile("" : "+f"(r[i]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(float* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const float* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31};" ::"f"(r[0]),
      "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]), "f"(r[10]),
      "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]), "f"(r[19]),
      "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]), "f"(r[26]), "f"(r[27]), "f"(r[28]),
      "f"(r[29]), "f"(r[30]), "f"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}

// 32 bytes to a 32-byte aligned address: a whole sector a thread.
__device__ __forceinline__ void stg256(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Pairs of floats in one 64-bit register: one instruction for two fp32 operations.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float lo2(f32x2 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi2(f32x2 v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Byte offset of 16-byte chunk c of key row r in a tile as it is in the pool, swizzled as
// the boxes are.
template <typename T>
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {
  constexpr int per = T::kRowB / 16;
  const uint32_t o = (c / per) * T::kSubB + r * T::kRowB + (c % per) * 16;
  return o ^ ((o >> 3) & T::kSwz);
}

// Byte offset of 16-byte chunk c of row r in a 16-bit tile of `rows` rows of 128 bytes
// per block of 64 values.
__device__ __forceinline__ uint32_t umma_offset(int rows, int r, int c) {
  return (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// What the warps of a CTA share besides tiles: barriers of the rings and hand-overs.
struct ChunkBars {
  uint64_t k_full[4], k_ready[4], k_empty[4];
  uint64_t v_full[4], v_ready[4], v_empty[4];
  uint64_t raw_full[4], raw_empty[4];
  uint64_t q_full[2];
  uint64_t s_full[2];             // one per group, or per S buffer
  uint64_t p_full[2][2];          // the same, for each half of the keys
  uint64_t o_full[2];             // products with V done: one per group, or in turn
  RangeScratch scratch;
  uint32_t tmem;
  int say[2];  // last_to_arrive's answers, by group
  NotedTiles noted;
};

// The infinities and NaN among 32 values of a pool (16-byte aligned), added to o: 16 bytes a
// load, as most of them hold none.
template <bool kFp8>
__device__ __forceinline__ void add_nonfinite(float (&o)[32], const void* pool, int64_t at) {
  if constexpr (kFp8) {
#pragma unroll
    for (int i = 0; i < 32; i += 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(pool) + at + i);
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if ((x[j / 4] >> (8 * (j % 4)) & 0x7f) == 0x7f) o[i + j] += __uint_as_float(0x7fffffff);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(pool) + at + i);
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = __uint_as_float(j % 2 ? x[j / 2] & 0xffff0000u : x[j / 2] << 16);
        if (!isfinite(f)) o[i + j] += f;
      }
    }
  }
}

// Infinities and NaN that were taken out of V in an item's n tiles from tile `tile0` of the
// CTA and key tile `first` on: from the pool into O of this thread's row, for the keys [see_lo, see_hi)
// that it sees.  Each lane looks at one key, then all of them at those that hold any in
// the columns at hand.  `head` is the offset of the kv head in a page.  (A function of its own
// that works on TMEM: inside the loop that writes the rows the mixed batch of 64-value heads took 146.0 us and
// 2,048 tokens over 32,768 E4M3 keys of 128 values 713, with it 145.4 and 710.)
template <int kDim, bool kFp8, int kKeys>
__device__ __noinline__ void restore_nonfinite(uint32_t o_at, const volatile NotedTiles* notes, uint32_t tile0, int n,
                                               int first, KeyRange kr, int see_lo, int see_hi, const int32_t* table,
                                               const void* pool, int64_t head, int64_t page_stride, int page_log2,
                                               int num_pages) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int c = 0; c < kDim; c += 32) {
    float o[32];
    tmem_ld32(o, o_at + c);
    tmem_loaded(o);
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const int key0 = (first + j) * kKeys;
      if (!notes->at(tile0 + j) || !partly_seen(kr, key0, kKeys)) continue;
      const int hi = min(key0 + kKeys, kr.any_hi);
#pragma unroll 1
      for (int k0 = max(key0, kr.any_lo); k0 < hi; k0 += 32) {
        int64_t at = 0;
        bool holds = false;
        if (k0 + lane < hi) {
          const int key = k0 + lane, page = __ldg(table + (key >> page_log2));
          at = page * page_stride + head + static_cast<int64_t>(key & ((1 << page_log2) - 1)) * kDim + c;
          holds = static_cast<unsigned>(page) < static_cast<unsigned>(num_pages) && holds_nonfinite<kFp8, 32>(pool, at);
        }
#pragma unroll 1
        for (unsigned left = __ballot_sync(0xffffffffu, holds); left; left &= left - 1) {
          const int who = __ffs(left) - 1, key = k0 + who;
          const int64_t from = __shfl_sync(0xffffffffu, at, who);
          if (key >= see_lo && key < see_hi) add_nonfinite<kFp8>(o, pool, from);
        }
      }
    }
    __syncwarp();  // the rows that see a key have gone their own way: TMEM is written by a whole warp
    tmem_st32(o_at + c, o);
  }
  tmem_wait_st();
}

// ------------------------------------------------------------------ the join of split items

// The join of a split item's shares, in groups of eight: the last holder of a group to
// arrive at its counter joins the group's shares in range order and goes on with the result
// as one of the next level's.  So nobody waits for another CTA, the result does not depend on
// the order of arrival, few shares take one step, and no CTA reads more than eight of
// them at a step.
constexpr int kJoinGroup = 8;

// One step up: shares [start, start + stride * kJoinGroup) of the item, `stride` apart
// (kJoinGroup ^ level).  Called by the kThreadsIn threads (named barrier `bar`) that have
// written share `mine`; true for the last to arrive, whose threads then see all of
// them.  Counters return to zero.
template <int kThreadsIn>
__device__ __forceinline__ bool last_to_arrive(unsigned* counter, int arrivals, int bar, volatile int* say) {
  __threadfence();
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(kThreadsIn) : "memory");
  if (threadIdx.x % kThreadsIn == 0) {
    const bool last = atomicAdd(counter, 1u) == static_cast<unsigned>(arrivals - 1);
    if (last) *counter = 0;
    *say = last;
  }
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(kThreadsIn) : "memory");
  const bool last = *say != 0;
  if (last) __threadfence();
  return last;
}

// A group of one has nothing to join and nobody to wait for: its share goes up a level without a
// counter.  With that, counters of different items never meet, although an item that ends
// in range c1 and the next one that starts there have shares of the same CTA: a group of
// two or more starts at least one share before its item's last, so that an item of shares c0 .. c1
// uses counters c0 .. c1 - 1, and the next one's begin at c1.  (The top group of a split item always has
// two or more.)
struct JoinStep {
  int start, stride, count, counter;  // shares start, start + stride, ... (count of them); the group's counter or -1
  bool top;                           // the item is whole after this step
};
__host__ __device__ __forceinline__ JoinStep join_step(int mine, int level, int holders) {
  JoinStep s;
  s.stride = level == 0 ? 1 : (level == 1 ? kJoinGroup : kJoinGroup * kJoinGroup);
  const int size = s.stride * kJoinGroup;
  s.start = mine / size * size;
  s.count = min(kJoinGroup, (holders - s.start + s.stride - 1) / s.stride);
  // distinct over groups and levels (start is a multiple of 8 ^ (level + 1)), and below the item's last
  // share: a group of two or more has its second one at start + 8 ^ level
  s.counter = s.count > 1 ? s.start + level : -1;
  s.top = size >= holders;
  return s;
}

// ------------------------------------------------------------------ the kernel

template <int kDim, bool kFp8>
__global__ void __launch_bounds__(ChunkTile<kDim, kFp8>::kThreadsAll, 1)
    attn_chunk_kernel(const AttnJob p, const __grid_constant__ KvMaps maps) {
  using T = ChunkTile<kDim, kFp8>;
  using KRing = typename T::KRing;
  using VRing = typename T::VRing;
  using RawRing = typename T::RawRing;
  constexpr int kG = T::kGroups, kKeys = T::kKeys;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw0 = smem_addr(smem_raw);
  const uint32_t base = (raw0 + 1023u) & ~1023u;
  ChunkBars* bars = reinterpret_cast<ChunkBars*>(smem_raw + (base - raw0) + T::kBars);
  static_assert(sizeof(ChunkBars) <= 1024, "barriers");
  const uint32_t q_at = base, k_at = base + T::kKAt, v_at = base + T::kVAt, raw_at = base + T::kRaw;

  const int warp = static_cast<int>(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(bars->k_full + i, 1), mbar_init(bars->k_ready + i, T::kFits), mbar_init(bars->k_empty + i, 1);
      mbar_init(bars->v_full + i, 1), mbar_init(bars->v_ready + i, T::kFits), mbar_init(bars->v_empty + i, 1);
      mbar_init(bars->raw_full + i, 1), mbar_init(bars->raw_empty + i, T::kFits);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars->q_full + i, 4), mbar_init(bars->s_full + i, 1);
      mbar_init(&bars->p_full[i][0], 4), mbar_init(&bars->p_full[i][1], 4);
      mbar_init(bars->o_full + i, 1);
    }
    fence_mbar_init();
  }
  bars->noted.clear(threadIdx.x);
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&bars->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*static_cast<volatile uint32_t*>(&bars->tmem));

  constexpr Tiling kTiling = T::tiling();
  Found f;
  Ranges ranges;
  find_range<T::kThreadsAll>(p, kTiling, gridDim.x, blockIdx.x, &ranges, &f, &bars->scratch,
                             reinterpret_cast<longlong2*>(smem_raw + (base - raw0)));
  // (the list lies where the first tiles will: its last reads come before the copies)
  fence_proxy_async_smem();
  __syncthreads();
  const bool idle = static_cast<int>(blockIdx.x) >= ranges.grid;
  const long long u0 = idle ? 0 : ranges.start(blockIdx.x), u1 = idle ? 0 : ranges.start(blockIdx.x + 1);
  Walk w;
  w.b = f.seq, w.item0 = f.before;
  if (!idle) walk_seq(p, w, kTiling);
  bool ran_out = false;  // a wait reached its limit (recorded): no further waits, the roles stay in step
#define NVFP4_WAIT(bar, parity) ran_out = ran_out || !mbar_wait_warp(bar, parity)

  // tile counts over all items so far: ring positions and phases
  uint32_t nt = 0;
  // Registers: with two softmax warpgroups the others give theirs to them (the shares add up to
  // what the block was launched with: 384 * 168 = 128 * (72 + 2 * 216), 512 * 128 = 128 * (64 + 64 + 2 * 192))
  if (warp < T::kSoft0) {
    if constexpr (kG == 2 && !T::kFitGroup) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if constexpr (kG == 2 && T::kFitGroup) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
      // ------------------------------------------------------------ copies
      const int piece_log2 = min(p.page_log2, log2c(kKeys));
      constexpr int kMostPieces = kKeys / 16;
      const int pieces = kKeys >> piece_log2;  // of a tile: at most kMostPieces
      uint32_t raw = 0, k_tiles = 0, v_tiles = 0;  // copied so far
      for (long long u = u0; u < u1 && !ran_out;) {
        walk_to(p, w, u, kTiling);
        const Share pc = share_at(w, u, u0, u1, blockIdx.x, kTiling);
        u = pc.end;
        const int n = static_cast<int>(uniform(pc.n)), head = static_cast<int>(uniform(w.h));
        if (n == 0) continue;
        const int32_t* table = p.table + static_cast<int64_t>(w.b) * p.max_pages;
        // lane i holds the page of piece i of a tile, looked up a tile ahead of its K
        const auto look_up = [&](int j) {
          return lane < pieces && j < n ? piece_page(p, table, (pc.first + j) * pieces + lane, piece_log2, w.t) : -1;
        };
        int page_k = look_up(0), page_v = page_k, page_next = look_up(1);
        // order: K 0, then K j + 1 and V j
        for (int c = 0; c < 2 * n; ++c) {
          const bool is_v = c == 2 * n - 1 || (c > 0 && c % 2 == 0);
          const int j = c == 0 ? 0 : (is_v ? (c == 2 * n - 1 ? n - 1 : c / 2 - 1) : (c + 1) / 2);
          const uint32_t g = nt + j;  // of its own ring
          uint64_t* full;
          uint32_t dst;
          if constexpr (kFp8) {
            const uint32_t st = RawRing::at(raw);
            if (RawRing::reused(raw)) NVFP4_WAIT(bars->raw_empty + st, RawRing::before(raw));
            full = bars->raw_full + st;
            dst = raw_at + st * T::kRawB;
          } else {
            const uint32_t st = is_v ? VRing::at(g) : KRing::at(g);
            if (is_v ? VRing::reused(g) : KRing::reused(g))
              NVFP4_WAIT((is_v ? bars->v_empty : bars->k_empty) + st, is_v ? VRing::before(g) : KRing::before(g));
            full = (is_v ? bars->v_full : bars->k_full) + st;
            dst = (is_v ? v_at : k_at) + st * T::kTileB;
          }
          if (ran_out) break;  // the place is still in use: no further copies
          ++raw;
          (is_v ? v_tiles : k_tiles) = g + 1;
          if (!is_v && c > 0) {
            page_v = page_k, page_k = page_next;
            page_next = look_up(j + 1);
          }
          const int page = is_v && c == 2 * n - 1 ? page_k : (is_v ? page_v : page_k);
          const uint32_t bar = smem_addr(full);
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, page >= 0)) << piece_log2 << log2c(T::kRowB * T::kSub);
          int at[kMostPieces];  // all pieces' pages first, then the copies back to back
#pragma unroll
          for (int i = 0; i < kMostPieces; ++i) at[i] = __shfl_sync(0xffffffffu, page, i);
          if (elect_one()) {
            mbar_arrive_expect_tx_s(bar, bytes);
#pragma unroll
            for (int i = 0; i < kMostPieces; ++i) {
              if (i >= pieces) break;
              if (at[i] < 0) continue;
              const int key = (pc.first + j) * kKeys + (i << piece_log2);
#pragma unroll
              for (int sub = 0; sub < T::kSub; ++sub)
                tma_load_5d(dst + sub * T::kSubB + (i << piece_log2) * T::kRowB, is_v ? &maps.v : &maps.k, 0,
                            key & ((1 << p.page_log2) - 1), sub, head, at[i], bar);
            }
          }
          __syncwarp();
        }
        nt += n;
      }
      // the CTA's shared memory is its own until its last copies have landed, whatever ran out (bounded)
      const auto land = [&](uint64_t* full, uint32_t tiles, auto ring) {
        using R = decltype(ring);
        for (uint32_t t = R::reused(tiles) ? tiles - R::kStages : 0; t < tiles; ++t)
          (void)mbar_wait_warp(full + R::at(t), R::phase(t));
      };
      if constexpr (kFp8)
        land(bars->raw_full, raw, RawRing{});
      else
        land(bars->k_full, k_tiles, KRing{}), land(bars->v_full, v_tiles, VRing{});
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issue
      const uint32_t id_qk = umma_idesc(!kFp8, false, kKeys, 128) | (p.scale < 0.f ? kNegateA : 0u);
      const uint32_t id_pv = umma_idesc(!kFp8, true, kDim, 128);
      uint32_t nq[2] = {0, 0}, np[2] = {0, 0};  // completed hand-overs of Q and P per group (or P per S buffer)
      // descriptors: the start address is the low 14 bits, in units of 16 bytes
      const uint64_t q_desc = umma_desc(q_at, 16, 1024), k_desc = umma_desc(k_at, 16, 1024);
      const uint64_t v_desc = umma_desc(v_at, kKeys * 128, 1024);
      const auto qk = [&](int g, uint32_t t) {
        const uint32_t d = tmem + T::kSCol + (kG == 2 ? g : (t & 1)) * kKeys;
        const uint64_t a = q_desc + g * (T::kQB >> 4), b = k_desc + KRing::at(t) * (T::kTileB >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kDim / 16; ++k)
            umma_ss(d, a + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4),
                    b + (((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4), id_qk, k > 0);
          umma_commit(bars->s_full + (kG == 2 ? g : (t & 1)));
        }
        __syncwarp();
      };
      const auto pv = [&](int g, uint32_t t, int half, bool add) {
        const uint32_t a = tmem + T::kSCol + (kG == 2 ? g : (t & 1)) * kKeys;
        const uint64_t b = v_desc + VRing::at(t) * (T::kTileB >> 4);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kKeys / 32; ++i) {
            const int k = half * (kKeys / 32) + i;
            umma_ts(tmem + g * kDim, a + 8 * k, b + k * (2048 >> 4), id_pv, add || i > 0);
          }
          if (half == 1) umma_commit(bars->o_full + (kG == 2 ? g : (t & 1)));
        }
        __syncwarp();
      };
      const auto free_tile = [&](uint64_t* bar) {
        if (elect_one()) umma_commit(bar);
        __syncwarp();
      };
      const auto wait_k = [&](uint32_t t) {
        NVFP4_WAIT((kFp8 ? bars->k_ready : bars->k_full) + KRing::at(t), KRing::phase(t));
      };
      for (long long u = u0; u < u1;) {
        walk_to(p, w, u, kTiling);
        const Share pc = share_at(w, u, u0, u1, blockIdx.x, kTiling);
        u = pc.end;
        const int n = static_cast<int>(uniform(pc.n));
        if (n == 0) continue;
        const int groups = kG == 2 && uniform(w.t.rows) > 128 ? 2 : 1;
        for (int g = 0; g < groups; ++g) {
          NVFP4_WAIT(bars->q_full + g, nq[g] & 1);
          ++nq[g];
        }
        wait_k(nt);
        tc_fence_after();
        for (int g = 0; g < groups; ++g) qk(g, nt);
        free_tile(bars->k_empty + KRing::at(nt));
        for (int j = 0; j < n; ++j) {
          const uint32_t t = nt + j;
          if (kG == 1 && j + 1 < n) {
            wait_k(t + 1);
            tc_fence_after();
            qk(0, t + 1);
            free_tile(bars->k_empty + KRing::at(t + 1));
          }
          NVFP4_WAIT(bars->v_ready + VRing::at(t), VRing::phase(t));
          if constexpr (!kFp8) NVFP4_WAIT(bars->v_full + VRing::at(t), VRing::phase(t));
          if (kG == 2 && j + 1 < n) wait_k(t + 1);
          for (int g = 0; g < groups; ++g) {
            const int pb = kG == 2 ? g : (t & 1);
            NVFP4_WAIT(&bars->p_full[pb][0], np[pb] & 1);
            tc_fence_after();
            pv(g, t, 0, j > 0);
            NVFP4_WAIT(&bars->p_full[pb][1], np[pb] & 1);
            ++np[pb];
            tc_fence_after();
            pv(g, t, 1, true);
            if (kG == 2 && j + 1 < n) qk(g, t + 1);
          }
          free_tile(bars->v_empty + VRing::at(t));
          if (kG == 2 && j + 1 < n) free_tile(bars->k_empty + KRing::at(t + 1));
        }
        nt += n;
      }
    } else if (warp >= T::kFit0) {
      // ------------------------------------------------------------ tiles made fit
      constexpr int kWho = 32 * T::kFits;
      const int who = (warp - T::kFit0) * 32 + lane;
      uint32_t raw = 0;
      for (long long u = u0; u < u1;) {
        walk_to(p, w, u, kTiling);
        const Share pc = share_at(w, u, u0, u1, blockIdx.x, kTiling);
        u = pc.end;
        if (pc.n == 0) continue;
        const int first = pc.first, n = pc.n;
        const KeyRange kr = key_range(p, w);
        if constexpr (!kFp8) {
          for (int j = 0; j < n; ++j) {
            const uint32_t t = nt + j, st = VRing::at(t);
            NVFP4_WAIT(bars->v_full + st, VRing::phase(t));
            const int key0 = (first + j) * kKeys;
            if (partly_seen(kr, key0, kKeys)) {
              const uint32_t tile = v_at + st * T::kTileB;
              bool noted = false;
              for (int r = who; r < kKeys; r += kWho) {
                const bool seen = key0 + r >= kr.any_lo && key0 + r < kr.any_hi;
#pragma unroll 1
                for (int c0 = 0; c0 < kDim / 8; c0 += 8) {  // (eight loads in flight)
                  uint4 v[8];
#pragma unroll
                  for (int c = 0; c < 8; ++c) v[c] = lds128(tile + umma_offset(kKeys, r, c0 + c));
#pragma unroll
                  for (int c = 0; c < 8; ++c)
                    sts128(tile + umma_offset(kKeys, r, c0 + c), clean_chunk<false>(v[c], seen, noted));
                }
              }
              if (noted) bars->noted.note(t);
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bars->v_ready + st);
          }
        } else {
          for (int c = 0; c < 2 * n; ++c, ++raw) {
            const bool is_v = c == 2 * n - 1 || (c > 0 && c % 2 == 0);
            const int j = c == 0 ? 0 : (is_v ? (c == 2 * n - 1 ? n - 1 : c / 2 - 1) : (c + 1) / 2);
            const uint32_t t = nt + j, st = is_v ? VRing::at(t) : KRing::at(t), rst = RawRing::at(raw);
            NVFP4_WAIT(bars->raw_full + rst, RawRing::phase(raw));
            if (is_v ? VRing::reused(t) : KRing::reused(t))
              NVFP4_WAIT((is_v ? bars->v_empty : bars->k_empty) + st, is_v ? VRing::before(t) : KRing::before(t));
            const int key0 = (first + j) * kKeys;
            const bool clean = is_v && partly_seen(kr, key0, kKeys);
            const uint32_t from = raw_at + rst * T::kRawB, to = (is_v ? v_at : k_at) + st * T::kTileB;
            bool noted = false;
            const auto convert = [&](auto cleaning) {
#pragma unroll 1
              for (int r = who; r < kKeys; r += kWho) {
                const bool seen = key0 + r >= kr.any_lo && key0 + r < kr.any_hi;
#pragma unroll 1
                for (int x0 = 0; x0 < kDim / 16; x0 += 4) {  // (four loads in flight)
                  uint4 v[4];
#pragma unroll
                  for (int x = 0; x < 4; ++x) v[x] = lds128(from + tile_offset<T>(r, x0 + x));
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    if constexpr (decltype(cleaning)::value) v[x] = clean_codes(v[x], seen, noted);
                    uint4 a, b;
                    e4m3x4_to_f16x2(v[x].x, a.x, a.y);
                    e4m3x4_to_f16x2(v[x].y, a.z, a.w);
                    e4m3x4_to_f16x2(v[x].z, b.x, b.y);
                    e4m3x4_to_f16x2(v[x].w, b.z, b.w);
                    sts128(to + umma_offset(kKeys, r, 2 * (x0 + x)), a);
                    sts128(to + umma_offset(kKeys, r, 2 * (x0 + x) + 1), b);
                  }
                }
              }
            };
            if (clean)
              convert(std::true_type{});
            else
              convert(std::false_type{});
            if (noted) bars->noted.note(t);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bars->raw_empty + rst);
              mbar_arrive((is_v ? bars->v_ready : bars->k_ready) + st);
            }
          }
        }
        nt += n;
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    if constexpr (kG == 2 && !T::kFitGroup) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    if constexpr (kG == 2 && T::kFitGroup) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int g = (warp - T::kSoft0) >> 2;
    const int row = (warp & 3) * 32 + lane;              // of the group: its TMEM lane
    const uint32_t lane_at = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_at = tmem + lane_at + g * kDim;
    const float log2e = 1.4426950408889634f;
    const float kOffset = kFp8 ? 7.0f : 0.0f;
    uint32_t mine = 0;  // this group's tiles so far
    // Q of this thread's row of the walk's item: copied as it is into the tile that the
    // products with K read
    const auto fetch_q = [&](const Walk& o) {
      const int r = g * 128 + row;
      const int rr = o.t.row0 + min(r, o.t.rows - 1);
      const int tok = div_by(p.by_group, rr), head = o.h * p.group + rr - tok * p.group;
      const uint16_t* q = p.q + (o.s.tok0 + tok) * p.q_stride + static_cast<int64_t>(head) * kDim;
      const uint32_t bytes = r < o.t.rows ? 16 : 0;  // rows past the tile's last one: zeros
#pragma unroll 8
      for (int c = 0; c < kDim / 8; ++c)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(q_at + g * T::kQB + umma_offset(128, row, c)),
                     "l"(q + 8 * c), "r"(bytes)
                     : "memory");
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // hands the copied tile over; for an E4M3 cache scaled by a power of two into f16's range.
    // Returns the factor that undoes the scaling.
    const auto hand_q = [&]() {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      if (p.scale == 0.f) {
#pragma unroll 1
        for (int c = 0; c < kDim / 8; ++c) {
          const uint32_t at = q_at + g * T::kQB + umma_offset(128, row, c);
          sts128(at, zero_or_nan(lds128(at)));
        }
      }
      float back = 1.0f;
      if constexpr (kFp8) {
        float amax = 0.f;
#pragma unroll 8
        for (int c = 0; c < kDim / 8; ++c) {
          const uint4 v = lds128(q_at + g * T::kQB + umma_offset(128, row, c));
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(x[i] & 0xffff0000u))));
        }
        const int e = pow2_rescale_exponent(amax);
        const float up = exp2i(e);
        back = exp2i(-e);
#pragma unroll 8
        for (int c = 0; c < kDim / 8; ++c) {
          const uint32_t at = q_at + g * T::kQB + umma_offset(128, row, c);
          const uint4 v = lds128(at);
          uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = f32x2_to_f16x2(__uint_as_float(x[i] << 16) * up, __uint_as_float(x[i] & 0xffff0000u) * up);
          sts128(at, make_uint4(x[0], x[1], x[2], x[3]));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars->q_full + g);
      return back;
    };

    float qscale = 1.0f;
    bool ready = false;  // Q of the walk's item has been handed over already
    for (long long u = u0; u < u1;) {
      walk_to(p, w, u, kTiling);
      const Share pc = share_at(w, u, u0, u1, blockIdx.x, kTiling);
      u = pc.end;
      if (pc.n == 0) continue;
      const int first = pc.first, n = pc.n;
      if (g * 128 >= w.t.rows) {  // this group has no rows here
        nt += n;
        continue;
      }
      if (!ready) {
        fetch_q(w);
        qscale = hand_q();
      }
      ready = false;
      const int r = g * 128 + row;
      const bool live = r < w.t.rows;
      const int rr = w.t.row0 + min(r, w.t.rows - 1);
      const int tok = div_by(p.by_group, rr), head = w.h * p.group + rr - tok * p.group;
      const int pos = w.s.len - w.s.n + tok;
      const int64_t token = w.s.tok0 + tok;
      const float ks = (kFp8 && p.k_scale) ? __ldg(p.k_scale + w.h) : 1.0f;
      const bool capped = p.softcap > 0.f;
      const float scale = fabsf(p.scale);  // its sign is in the product
      // logits in units of log 2: s * mul; with a softcap, mul * tanh(s * unit)
      const float unit = scale * ks * qscale * (capped ? 1.0f / p.softcap : log2e);
      const float mul = fmaxf(capped ? p.softcap * log2e : unit, 1.2e-38f);  // (-inf * 0 would be NaN)
      // keys that this row sees, and those that all rows of the warp see
      const int see_hi = min(pos + 1, w.s.len), see_lo = p.window > 0 ? pos - p.window + 1 : -(1 << 30);

      float m = -INFINITY, l = 0.f;  // reference of the weights, this row's sum
      for (int j = 0; j < n; ++j, ++mine) {
        const uint32_t t = nt + j;
        const int sb = kG == 2 ? g : (t & 1);
        NVFP4_WAIT(bars->s_full + sb, (kG == 2 ? mine : (t >> 1)) & 1);
        tc_fence_after();
        const uint32_t s_at = tmem + lane_at + T::kSCol + sb * kKeys;
        const int key0 = (first + j) * kKeys;
        const bool partly = __any_sync(0xffffffffu, key0 + kKeys > see_hi || key0 < see_lo);
        if (partly || capped) {
          // in TMEM, before the rest reads it: two paths of tanh over a whole row would cost every
          // other call registers (a prompt of 4,096 tokens 140 us instead of 137)
#pragma unroll 1
          for (int c = 0; c < kKeys; c += 32) {
            float x[32], high = 0.f;
            tmem_ld32(x, s_at + c);
            tmem_loaded(x);
            if (capped) {
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] *= unit, high = fmaxf(high, fabsf(x[i]));
              if (__any_sync(0xffffffffu, high >= kTanhSmall)) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = tanh_any(x[i]);
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = tanh_small(x[i]);
              }
            }
            if (partly) {
              const int hi = see_hi - key0 - c, lo = see_lo - key0 - c;
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = i >= lo && i < hi ? x[i] : -INFINITY;
            }
            tmem_st32(s_at + c, x);
          }
          tmem_wait_st();
        }
        float s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld32(s + c, s_at + c);
        tmem_loaded(s);
        float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c + 8 <= kKeys; c += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) top[i] = max3(top[i], s[c + i], s[c + 4 + i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = fmaxf(top[i], s[kKeys - 4 + i]);
        const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * mul - kOffset;
        const bool move = high > m + 8.0f || m == -INFINITY;
        if (__any_sync(0xffffffffu, move && j > 0 && high > m)) {
          // the row's sums follow its maximum: everything up to the tile before is in O
          if constexpr (kG == 1) {
            NVFP4_WAIT(bars->o_full + ((t - 1) & 1), ((t - 1) >> 1) & 1);
            tc_fence_after();
          }
          const float a = move && high > m ? exp2_approx(m - high) : 1.0f;
          l *= a;
#pragma unroll 1
          for (int c = 0; c < kDim; c += 32) {
            float o[32];
            tmem_ld32(o, o_at + c);
            tmem_loaded(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= a;
            tmem_st32(o_at + c, o);
          }
          tmem_wait_st();
        }
        if (move && high > m) m = high;
        const float ref = m == -INFINITY ? 0.f : m;
        // weights, handed over in two halves: the product with V starts on the first one
        const f32x2 mul2 = pack2(mul, mul), ref2 = pack2(-ref, -ref);
        f32x2 sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int c = half * kKeys / 2; c < (half + 1) * kKeys / 2; c += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const f32x2 e = fma2(pack2(s[c + 2 * i], s[c + 2 * i + 1]), mul2, ref2);
              const float a = exp2_approx(lo2(e)), b = exp2_approx(hi2(e));
              sum[i & 1] = add2(sum[i & 1], pack2(a, b));
              pk[i] = kFp8 ? f32x2_to_f16x2(a, b) : f32x2_to_bf16x2(a, b);
            }
            tmem_st16(s_at + c / 2, pk);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p_full[sb][half]);
        }
        const f32x2 both = add2(sum[0], sum[1]);
        l += lo2(both) + hi2(both);
      }
      nt += n;

      // ---- the next item's Q while the last product with V runs (all products with this
      // item's Q are done: their last S has been read)
      Walk next = w;
      bool more = false;
      for (long long v = u; v < u1 && !more;) {
        walk_to(p, next, v, kTiling);
        const Share q = share_at(next, v, u0, u1, blockIdx.x, kTiling);
        more = q.n > 0;
        v = q.end;
      }
      more = more && g * 128 < next.t.rows;
      if (more) fetch_q(next);

      // ---- write: the finished row, or this piece's share of it
      if constexpr (kG == 2)
        NVFP4_WAIT(bars->o_full + g, (mine - 1) & 1);
      else
        NVFP4_WAIT(bars->o_full + ((nt - 1) & 1), ((nt - 1) >> 1) & 1);
      tc_fence_after();
      const bool whole = pc.whole;
      const int slot = pc.slot;
      const float vs = (kFp8 && p.v_scale) ? __ldg(p.v_scale + w.h) : 1.0f;
      const float inv = !whole ? 1.0f : (l == 0.f ? 0.f : vs / l);
      const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0 && (p.out_stride & 15) == 0;
      uint16_t* out = p.out + token * p.out_stride + static_cast<int64_t>(head) * kDim;
      // blocks of eight columns of all rows: neighbouring threads write neighbouring addresses
      float* part = p.part + static_cast<int64_t>(slot) * T::kRows * kDim + r * 8;
      const auto write_out = [&](const float (&o)[32], int c, float unit_out) {  // columns [c, c + 32) of this row
        if (!live) return;
        uint32_t x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = f32x2_to_bf16x2(o[2 * i] * unit_out, o[2 * i + 1] * unit_out);
        if (wide) {
          stg256(out + c, x);
          stg256(out + c + 16, x + 8);
        } else {
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<uint4*>(out + c + 2 * i) = make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        }
      };
      if (bars->noted.any_since(nt - n))
        restore_nonfinite<kDim, kFp8, kKeys>(o_at, &bars->noted, nt - n, n, first, key_range(p, w), see_lo, see_hi,
                                             p.table + static_cast<int64_t>(w.b) * p.max_pages, p.v_pool,
                                             value_at(p, 0, w.h, 0, kDim), p.page_stride, p.page_log2, p.num_pages);
#pragma unroll 1
      for (int c = 0; c < kDim; c += 32) {
        float o[32];
        tmem_ld32(o, o_at + c);
        tmem_loaded(o);
        if (c == 0 && more) {  // the next item's first product may start
          tc_fence_before();
          qscale = hand_q();
          ready = true;
        }
        if (whole) {
          write_out(o, c, inv);
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            stg256(part + static_cast<int64_t>((c + i) / 8) * T::kRows * 8, reinterpret_cast<const uint32_t*>(o) + i);
        }
      }
      float* ml = p.part + static_cast<int64_t>(2) * gridDim.x * T::kRows * kDim;  // references and sums, after all shares
      if (!whole)
        *reinterpret_cast<float2*>(ml + (static_cast<int64_t>(slot) * T::kRows + r) * 2) = make_float2(m, l);
      else if (live && p.lse)
        p.lse[token * p.n_heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      // ---- the join's steps of a split item, for as long as this group is the last to arrive
      if (!pc.whole) {
        const Holders h = holders_of(w, ranges, kTiling);
        int mine = static_cast<int>(blockIdx.x) - h.c0;
        for (int level = 0;; ++level) {
          const JoinStep s = join_step(mine, level, h.c1 - h.c0 + 1);
          if (s.counter < 0) {
            mine = s.start;
            continue;
          }
          if (!last_to_arrive<128>(p.counters + 2 * (h.c0 + s.counter) + g, s.count, 1 + g, &bars->say[g])) break;
          const auto slot_of = [&](int i) {
            const int share = s.start + i * s.stride;
            return static_cast<int64_t>(2 * (h.c0 + share) + (share == 0));
          };
          float high = -INFINITY, all = 0.f;
          for (int i = 0; i < s.count; ++i) high = fmaxf(high, __ldcg(ml + (slot_of(i) * T::kRows + r) * 2));
          for (int i = 0; i < s.count; ++i) {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(ml + (slot_of(i) * T::kRows + r) * 2));
            all += v.y * (high == -INFINITY ? 1.0f : exp2_approx(v.x - high));
          }
          const float unit_out = !s.top ? 1.0f : (all == 0.f ? 0.f : vs / all);
          float* into = p.part + slot_of(0) * T::kRows * kDim + r * 8;
#pragma unroll 1
          for (int c0 = 0; c0 < kDim; c0 += 32) {
            float o[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.f;
#pragma unroll 2
            for (int c = 0; c < s.count; ++c) {
              const int64_t at = slot_of(c);
              const float v = __ldcg(ml + (at * T::kRows + r) * 2);
              const float a = high == -INFINITY ? 1.0f : exp2_approx(v - high);
              const float4* x = reinterpret_cast<const float4*>(p.part + at * T::kRows * kDim +
                                                                (static_cast<int64_t>(c0 / 8) * T::kRows + r) * 8);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 y = __ldcg(x + (i / 2) * T::kRows * 2 + (i & 1));
                o[4 * i] += a * y.x, o[4 * i + 1] += a * y.y, o[4 * i + 2] += a * y.z, o[4 * i + 3] += a * y.w;
              }
            }
            if (s.top)
              write_out(o, c0, unit_out);
            else
#pragma unroll
              for (int i = 0; i < 32; i += 8)
                stg256(into + static_cast<int64_t>((c0 + i) / 8) * T::kRows * 8, reinterpret_cast<const uint32_t*>(o) + i);
          }
          if (s.top) {
            if (live && p.lse)
              p.lse[token * p.n_heads + head] = all == 0.f ? -INFINITY : (high + log2f(all)) * 0.6931471805599453f;
            break;
          }
          *reinterpret_cast<float2*>(ml + (slot_of(0) * T::kRows + r) * 2) = make_float2(high, all);
          mine = s.start;  // the joined share takes the place of the group's first
        }
      }
      tc_fence_before();  // O has been read before the next item's first P is handed over
    }
  }
#undef NVFP4_WAIT
  if (ran_out) {  // products may still be under way: give them time to end before TMEM is given back
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <int kDim, bool kFp8>
nvfp4_status launch_attn_chunk(const AttnJob& p, const KvMaps& maps, cudaStream_t stream) {
  using T = ChunkTile<kDim, kFp8>;
  if (set_smem(attn_chunk_kernel<kDim, kFp8>, T::kSmem) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (launch_pdl(attn_chunk_kernel<kDim, kFp8>, dim3(kAttnGrid), dim3(T::kThreadsAll), T::kSmem, stream, p, maps) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  return launched();
}

}  // namespace nvfp4
