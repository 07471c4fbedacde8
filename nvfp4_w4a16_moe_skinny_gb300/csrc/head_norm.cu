// Norms of queries and keys for each head with rotary positions in the same pass
// (qk_norm_rope), on the way to a paged cache (kv_append_norm), and back
// (qk_norm_rope_backward).
//
// With the head's values x, weights g, r = 1 / sqrt(mean(x^2) + eps), R the rotation by a
// token's angles (which leaves the values past rot_dim alone) and A the amplitude:
//   y = A R (x r g).
// Back, with u = A R^T dy (the values past rot_dim: dy) and z = u g:
//   dx = r (z - x r mean(z x r)),   dg = sum over tokens and heads of u x r.
// Sums and products are fp32, each result rounded once.
//
// A thread holds 16 values of a head, 8 pairs, and walks heads with the same angles and weights; the lanes of a head
// share its sums by shuffles.  Bound by memory at prompt sizes: 8,191 tokens of 32 + 8 heads of 128
// values (168 MB) take 28.7 us, 5.8 TB/s or 86% of the rate of a plain copy, into an E4M3 cache with their values
// (185 MB) 31.9 us (85%), back (252 MB) 46.2 us (80%, 3 us of it the second grid, which sums the weights' gradients).  By the launch at
// decode sizes: 16 tokens 3.4 us, back 7.2 us.
#include <cmath>
#include <cstdint>

#include "rope.cuh"

namespace nvfp4 {
namespace {

constexpr int kNormThreads = 128;

struct NormJob {
  const uint16_t* x[3];      // rows of q, k, v (heads 0: none)
  int64_t x_stride[3];
  int heads[3];
  const uint16_t* dy[2];     // backward: rows of dq, dk
  int64_t dy_stride[2];
  uint16_t* y[2];            // rows of q and (without a cache) k; backward: their gradients
  int64_t y_stride[2];
  const void* weight[2];     // of q and k
  int weight_f32;
  float eps, inv_dim;
  uint8_t* cache[2];         // pools of k and v
  const float* scale[2];
  int64_t page_stride;       // elements
  int64_t n_slots;
  int page_log2;
  const int64_t* slots;
  const int32_t* positions;
  const double* inv_freq;
  float amplitude;
  int n_tokens, dim, rot;
  int lanes_log2;            // lanes of a head: its chunks of 16 values, rounded up to a power of two
  int per_thread;            // heads that one thread walks
  int groups[3];             // ceil(heads / per_thread)
  float* partial;            // backward: each block's share of dg, [blocks][dim]
};

// The 16 values of a thread as 8 pairs to turn, (a + i, b + i) or, where pairs interleave, (a + 2 i, a + 2 i + 1), two of
// them to a register pair: a[j] holds the first members of pairs 2 j and 2 j + 1, b[j] the second ones.
struct Pairs {
  f32x2 a[4], b[4];
};
__device__ __forceinline__ float low_half(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_half(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <bool kInterleaved>
__device__ __forceinline__ Pairs unpack_pairs(uint4 va, uint4 vb) {
  const uint32_t w[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
  Pairs p;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    p.a[j] = kInterleaved ? pack2(low_half(w[2 * j]), low_half(w[2 * j + 1])) : pack2(low_half(w[j]), high_half(w[j]));
    p.b[j] = kInterleaved ? pack2(high_half(w[2 * j]), high_half(w[2 * j + 1])) : pack2(low_half(w[4 + j]), high_half(w[4 + j]));
  }
  return p;
}
// back to runs of eight values
template <bool kInterleaved>
__device__ __forceinline__ void runs_of(const Pairs& p, float (&fa)[8], float (&fb)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (kInterleaved) {
      float* f = j < 2 ? fa + 4 * j : fb + 4 * j - 8;
      f[0] = lo2(p.a[j]), f[1] = lo2(p.b[j]), f[2] = hi2(p.a[j]), f[3] = hi2(p.b[j]);
    } else {
      fa[2 * j] = lo2(p.a[j]), fa[2 * j + 1] = hi2(p.a[j]);
      fb[2 * j] = lo2(p.b[j]), fb[2 * j + 1] = hi2(p.b[j]);
    }
  }
}

template <int kLanesLog2 = -1>
__device__ __forceinline__ float lanes_sum(float v, int lanes_log2) {
#pragma unroll
  for (int k = 0; k < 5; ++k)
    if (k < (kLanesLog2 >= 0 ? kLanesLog2 : lanes_log2)) v += __shfl_xor_sync(0xffffffffu, v, 1 << k);
  return v;
}

// A thread's own ring in shared memory, through which its loads of the next kAhead heads come without holding
// registers: 16-byte pieces, kParts a head, each read by the thread that copied it, so that no barrier is needed.
// A slot is filled again one head after it was read (a thread's own order: what it read is in registers by then).
template <int kParts>
struct OwnRing {
  static constexpr int kSlots = 4, kAhead = kSlots - 1, kBytes = kSlots * kParts * kNormThreads * 16;
  uint32_t base;
  __device__ __forceinline__ uint32_t at(int i, int part) const {
    return base + (((i & (kSlots - 1)) * kParts + part) * kNormThreads + threadIdx.x) * 16;
  }
  // 16 bytes, or zeros where `bytes` is 0 (nothing is read then)
  __device__ __forceinline__ void copy(int i, int part, const uint16_t* from, uint32_t bytes) const {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(i, part)), "l"(from), "r"(bytes) : "memory");
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  static __device__ __forceinline__ void arrived() { asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory"); }
  __device__ __forceinline__ uint4 read(int i, int part) const { return lds128(at(i, part)); }
};

// Whether mean(x^2) + eps is near an end of fp32: the squares of values above 2^60 may overflow, those of a
// head of very small ones (and eps) vanish.  Such a head is multiplied by scale_of and its sums taken again.
__device__ __forceinline__ bool out_of_range(float v) { return !(v > 0x1p-100f && v < 0x1p120f); }
__device__ __forceinline__ float scale_of(float v) { return v >= 1.0f ? 0x1p-80f : 0x1p80f; }

// What a thread holds of its head: two runs of eight values, and whether their pairs turn.  The runs of neighbouring
// lanes are neighbours, so that every access covers whole sectors: pairs that interleave are four to a run, the runs
// half a head apart; otherwise a run holds eight pairs' first members and the other, half a rotation on, their
// second ones, and past the rotated values the runs lie half of those apart.  (Both runs next to each other: the way back
// through 8,191 tokens with interleaved pairs 72.8 us, three times the sectors.)
struct Chunk {
  int token, a, b;
  bool inside, turn_a, turn_b;  // (turn_a and turn_b are one where pairs do not interleave)
};

template <bool kInterleaved>
__device__ __forceinline__ Chunk chunk_at(const NormJob& p, int token, int chunk) {
  Chunk h;
  h.token = min(token, p.n_tokens - 1);
  h.inside = token < p.n_tokens && chunk < (p.dim >> 4);
  if (kInterleaved) {
    h.a = 8 * chunk, h.b = h.a + (p.dim >> 1);
    h.turn_a = h.a < p.rot, h.turn_b = h.b < p.rot;
  } else {
    h.turn_a = h.turn_b = chunk < (p.rot >> 4);
    h.a = h.turn_a ? 8 * chunk : p.rot + 8 * (chunk - (p.rot >> 4));
    h.b = h.a + ((h.turn_a ? p.rot : p.dim - p.rot) >> 1);
  }
  if (chunk >= (p.dim >> 4)) h.a = h.b = 0;  // (a lane past the head: its copies are of nothing, from inside the row)
  return h;
}

// Place of the first members of pairs 2 j and 2 j + 1 among the head's values, from one to the next, and to the
// second ones; and the frequency of the first.
template <bool kInterleaved>
struct PairAt {
  int first, step, second, frequency;
  __device__ __forceinline__ PairAt(const Chunk& h, int j) {
    if (kInterleaved) {
      first = (j < 2 ? h.a + 4 * j : h.b + 4 * j - 8), step = 2, second = first + 1, frequency = first >> 1;
    } else {
      first = h.a + 2 * j, step = 1, second = h.b + 2 * j, frequency = first;
    }
  }
};

template <bool kInterleaved>
__device__ __forceinline__ Pairs load_weights(const NormJob& p, int kind, const Chunk& h) {
  const auto at = [&](int i) {
    if (p.weight_f32) return __ldg(static_cast<const float*>(p.weight[kind]) + i);
    return bf16_bits_to_f32(__ldg(static_cast<const uint16_t*>(p.weight[kind]) + i));
  };
  Pairs g{};
  if (!h.inside) return g;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const PairAt<kInterleaved> i(h, j);
    g.a[j] = pack2(at(i.first), at(i.first + i.step)), g.b[j] = pack2(at(i.second), at(i.second + i.step));
  }
  return g;
}

// cos and sin of a thread's pairs, times the amplitude, two of them to a register pair.
template <bool kInterleaved>
__device__ __forceinline__ void load_angles(const NormJob& p, const Chunk& h, f32x2 (&c)[4], f32x2 (&s)[4]) {
  if (!h.turn_a) return;  // (turn_b implies turn_a)
  const int pos = __ldg(p.positions + h.token);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (kInterleaved && j >= 2 && !h.turn_b) break;
    const PairAt<kInterleaved> i(h, j);
    float c0, c1, s0, s1;
    angle_of(p.inv_freq, p.amplitude, false, pos, i.frequency, c0, s0);
    angle_of(p.inv_freq, p.amplitude, false, pos, i.frequency + 1, c1, s1);
    c[j] = pack2(c0, c1), s[j] = pack2(s0, s1);
  }
}
// whether pairs 2 j and 2 j + 1 turn
template <bool kInterleaved>
__device__ __forceinline__ bool turns(const Chunk& h, int j) {
  return kInterleaved && j >= 2 ? h.turn_b : h.turn_a;
}

__device__ __forceinline__ f32x2 negative2(f32x2 v) { return v ^ 0x8000000080000000ull; }
__device__ __forceinline__ f32x2 both2(float v) { return pack2(v, v); }
__device__ __forceinline__ float sum2(f32x2 v) { return lo2(v) + hi2(v); }

// This thread's share of the head's sum of squares.
__device__ __forceinline__ float squares_of(const Pairs& x) {
  f32x2 s = mul2(x.a[0], x.a[0]), t = mul2(x.b[0], x.b[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) s = fma2(x.a[j], x.a[j], s), t = fma2(x.b[j], x.b[j], t);
  return sum2(add2(s, t));
}
__device__ __forceinline__ float products_of(const Pairs& u, const Pairs& g, const Pairs& x) {
  f32x2 s = mul2(mul2(u.a[0], g.a[0]), x.a[0]), t = mul2(mul2(u.b[0], g.b[0]), x.b[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) s = fma2(mul2(u.a[j], g.a[j]), x.a[j], s), t = fma2(mul2(u.b[j], g.b[j]), x.b[j], t);
  return sum2(add2(s, t));
}
__device__ __forceinline__ void scale_pairs(Pairs& x, float by) {
#pragma unroll
  for (int j = 0; j < 4; ++j) x.a[j] = mul2(x.a[j], both2(by)), x.b[j] = mul2(x.b[j], both2(by));
}

enum { kToRows = 0, kToBf16 = 1, kToE4M3 = 2 };  // where keys and values go

// (Registers for six blocks an SM: the prompt above 29.4 us, for seven 30.4, for eight, which spill, 34.0.  Eight slots of
// the ring at six blocks 29.1, and heads of 256 values 21.4 us instead of 20.6.)
template <int kTo, bool kInterleaved>
__global__ void __launch_bounds__(kNormThreads, 6) norm_rope_kernel(const NormJob p) {
  __shared__ __align__(16) uint8_t ring_bytes[OwnRing<2>::kBytes];
  const OwnRing<2> ring{smem_addr(ring_bytes)};
  pdl_wait();
  pdl_launch_dependents();
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x;
  const Chunk h = chunk_at<kInterleaved>(p, static_cast<int>(idx >> p.lanes_log2),
                                         static_cast<int>(idx) & ((1 << p.lanes_log2) - 1));
  int g = blockIdx.y, kind = 0;
  while (kind < 2 && g >= p.groups[kind]) g -= p.groups[kind++];
  const int h0 = g * p.per_thread, h1 = min(p.heads[kind], h0 + p.per_thread);
  const bool to_cache = kTo != kToRows && kind > 0;

  bool live = h.inside;
  int64_t slot = 0;
  if (to_cache) {
    slot = __ldg(p.slots + h.token);
    if (slot >= p.n_slots && live && h.a == 0) atomicOr(&g_device_error, kErrPage);
    live = live && slot >= 0 && slot < p.n_slots;
  }
  const uint16_t* x = p.x[kind] + h.token * p.x_stride[kind] + h0 * p.dim;
  const auto fetch = [&](int i) {
    if (h0 + i < h1) {
      ring.copy(i, 0, x + i * p.dim + h.a, live ? 16 : 0);
      ring.copy(i, 1, x + i * p.dim + h.b, live ? 16 : 0);
    }
    ring.commit();
  };
#pragma unroll
  for (int i = 0; i < ring.kAhead; ++i) fetch(i);
  // with n = x r a turned pair is (na ga c - nb gb s, nb gb c + na ga s): the weights are multiplied in once for all heads
  // (and r first: x g may leave fp32's range where n g does not)
  Pairs along{}, across{};
  if (kind < 2) {
    along = load_weights<kInterleaved>(p, kind, h);
    f32x2 c[4], s[4];
    load_angles<kInterleaved>(p, h, c, s);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (turns<kInterleaved>(h, j)) {
        across.a[j] = mul2(along.a[j], s[j]), across.b[j] = negative2(mul2(along.b[j], s[j]));
        along.a[j] = mul2(along.a[j], c[j]), along.b[j] = mul2(along.b[j], c[j]);
      }
    }
  }
  // element offset of (slot, head 0) in a pool, and from one head to the next
  const int64_t page = slot >> p.page_log2, off = slot & ((1 << p.page_log2) - 1);
  const int64_t base = to_cache ? page * p.page_stride + off * p.dim : h.token * p.y_stride[kind < 2 ? kind : 0];
  const int64_t head_step = to_cache ? static_cast<int64_t>(p.dim) << p.page_log2 : p.dim;
  uint16_t* const y = to_cache ? reinterpret_cast<uint16_t*>(p.cache[kind - 1]) : p.y[kind < 2 ? kind : 0];
  for (int hh = h0; hh < h1; ++hh) {
    ring.arrived();
    const uint4 va = ring.read(hh - h0, 0), vb = ring.read(hh - h0, 1);
    fetch(hh - h0 + ring.kAhead);
    const int64_t o = base + hh * head_step;
    float fa[8], fb[8];
    if (kind == 2) {
      if (!live) continue;
      if (kTo != kToE4M3) {  // values are copied as they are
        *reinterpret_cast<uint4*>(y + o + h.a) = va;
        *reinterpret_cast<uint4*>(y + o + h.b) = vb;
        continue;
      }
      unpack8(va, fa);
      unpack8(vb, fb);
    } else {
      Pairs x = unpack_pairs<kInterleaved>(va, vb);
      float v = fmaf(lanes_sum(squares_of(x), p.lanes_log2), p.inv_dim, p.eps);
      const bool odd = out_of_range(v);
      if (__any_sync(0xffffffffu, odd)) {
        const float unit = odd ? scale_of(v) : 1.0f;
        scale_pairs(x, unit);
        v = fmaf(lanes_sum(squares_of(x), p.lanes_log2), p.inv_dim, p.eps * unit * unit);
      }
      const f32x2 r = both2(rsqrtf(v));
      if (!live) continue;  // (the shuffles are done: the next head's are taken by all lanes again)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 na = mul2(x.a[j], r), nb = mul2(x.b[j], r);
        x.a[j] = mul2(na, along.a[j]), x.b[j] = mul2(nb, along.b[j]);
        if (turns<kInterleaved>(h, j)) x.a[j] = fma2(nb, across.b[j], x.a[j]), x.b[j] = fma2(na, across.a[j], x.b[j]);
      }
      runs_of<kInterleaved>(x, fa, fb);
    }
    if (kTo == kToE4M3 && to_cache) {
      const HeadScale sc = head_scale(p.scale[kind - 1] ? __ldg(p.scale[kind - 1] + hh) : 1.0f);
      *reinterpret_cast<uint2*>(p.cache[kind - 1] + o + h.a) = pack8_e4m3(fa, sc);
      *reinterpret_cast<uint2*>(p.cache[kind - 1] + o + h.b) = pack8_e4m3(fb, sc);
    } else {
      *reinterpret_cast<uint4*>(y + o + h.a) = pack8(fa);
      *reinterpret_cast<uint4*>(y + o + h.b) = pack8(fb);
    }
  }
}

// Each block takes a contiguous range of units, all of them of a size: one head of the tokens that the block holds at once.
// They are numbered by kind (queries, then keys), tokens, heads, so that a block walks the heads of its tokens with the
// same angles and changes from queries to keys at most once.
struct BackwardUnits {
  int per_block, blocks;      // units of a block (the last one may have fewer)
  int64_t of_q, all;
  int shares_q, shares_k;     // blocks with units of q, of k
  int first_k;                // the first of the latter
};

// kLanesLog2: lanes of a head whose chunks fill them (64, 128 and 256 values), or -1: any head.  (Registers and ring for
// four blocks an SM, with an earlier second grid: 47.2 us; for three 54.8, for five, which spill, 67.5; eight slots of the ring, three blocks, 58.7.)
template <bool kInterleaved, int kLanesLog2>
__global__ void __launch_bounds__(kNormThreads, 4) norm_rope_backward_kernel(const NormJob p, const BackwardUnits units) {
  __shared__ __align__(16) uint8_t ring_bytes[OwnRing<4>::kBytes];
  __shared__ float sums[kNormThreads * 16];  // [tokens of the block][dim]
  const OwnRing<4> ring{smem_addr(ring_bytes)};
  pdl_wait();
  pdl_launch_dependents();
  const int lanes_log2 = kLanesLog2 >= 0 ? kLanesLog2 : p.lanes_log2, dim = kLanesLog2 >= 0 ? 16 << kLanesLog2 : p.dim;
  const int at_once = kNormThreads >> lanes_log2;
  const int sub = threadIdx.x >> lanes_log2, chunk = threadIdx.x & ((1 << lanes_log2) - 1);
  int64_t u = static_cast<int64_t>(blockIdx.x) * units.per_block;
  const int64_t end = min(u + units.per_block, units.all);
  int kind = u >= units.of_q ? 1 : 0;
  const int64_t nth = kind ? u - units.of_q : u;
  const int64_t step0 = nth / p.heads[kind];
  int token0 = static_cast<int>(step0) * at_once, head = static_cast<int>(nth - step0 * p.heads[kind]);

  // the copies run through the same units, ahead of the loop
  int to_copy = static_cast<int>(end - u), copied = 0, ahead_kind = kind, ahead_token0 = token0, ahead_left = 0;
  const uint16_t *x_from = nullptr, *dy_from = nullptr;
  uint32_t bytes = 0;
  const Chunk here = chunk_at<kInterleaved>(p, 0, chunk);  // (its runs are those of every token)
  const auto copy_from = [&](int first_head) {
    const int token = min(ahead_token0 + sub, p.n_tokens - 1);
    bytes = here.inside && ahead_token0 + sub < p.n_tokens ? 16 : 0;
    x_from = p.x[ahead_kind] + token * p.x_stride[ahead_kind] + first_head * dim;
    dy_from = p.dy[ahead_kind] + token * p.dy_stride[ahead_kind] + first_head * dim;
    ahead_left = p.heads[ahead_kind] - first_head;
  };
  copy_from(head);
  const auto fetch = [&]() {
    if (copied < to_copy) {
      ring.copy(copied, 0, x_from + here.a, bytes);
      ring.copy(copied, 1, x_from + here.b, bytes);
      ring.copy(copied, 2, dy_from + here.a, bytes);
      ring.copy(copied, 3, dy_from + here.b, bytes);
      ++copied;
      x_from += dim, dy_from += dim;
      if (--ahead_left == 0 && copied < to_copy) {  // the next tokens; after the last ones of q, k's first
        ahead_token0 += at_once;
        if (ahead_token0 >= p.n_tokens) ahead_kind = 1, ahead_token0 = 0;
        copy_from(0);
      }
    }
    ring.commit();
  };
#pragma unroll
  for (int i = 0; i < ring.kAhead; ++i) fetch();
  int at = 0;
  for (; u < end; kind = 1, token0 = 0, head = 0) {
    const Pairs g = load_weights<kInterleaved>(p, kind, here);
    Pairs acc{};
    const int64_t kind_end = kind ? end : min(end, units.of_q);
    for (; u < kind_end; token0 += at_once, head = 0) {
      const Chunk h = chunk_at<kInterleaved>(p, token0 + sub, chunk);
      f32x2 c[4], s[4];
      load_angles<kInterleaved>(p, h, c, s);
      uint16_t* dx = p.y[kind] + h.token * p.y_stride[kind] + head * dim;
      const int heads = static_cast<int>(min(static_cast<int64_t>(p.heads[kind] - head), kind_end - u));
      u += heads;
      for (const int last = at + heads; at < last; ++at, dx += dim) {
        ring.arrived();
        Pairs x = unpack_pairs<kInterleaved>(ring.read(at, 0), ring.read(at, 1));
        Pairs d = unpack_pairs<kInterleaved>(ring.read(at, 2), ring.read(at, 3));
        fetch();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!turns<kInterleaved>(h, j)) continue;
          const f32x2 t = fma2(d.b[j], s[j], mul2(d.a[j], c[j]));
          d.b[j] = fma2(d.a[j], negative2(s[j]), mul2(d.b[j], c[j]));
          d.a[j] = t;
        }
        float unit = 1.0f;
        float v = fmaf(lanes_sum<kLanesLog2>(squares_of(x), lanes_log2), p.inv_dim, p.eps);
        const bool odd = out_of_range(v);
        if (__any_sync(0xffffffffu, odd)) {
          unit = odd ? scale_of(v) : 1.0f;
          scale_pairs(x, unit);
          v = fmaf(lanes_sum<kLanesLog2>(squares_of(x), lanes_log2), p.inv_dim, p.eps * unit * unit);
        }
        // with n = x r: dx = r (z - n along), along = mean(z n)  (z x may leave fp32's range where z n does not)
        const float r = rsqrtf(v);
        scale_pairs(x, r);
        const float along = lanes_sum<kLanesLog2>(products_of(d, g, x), lanes_log2) * p.inv_dim;
        if (!h.inside) continue;
        const f32x2 r2 = both2(r), less2 = both2(-along);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc.a[j] = fma2(d.a[j], x.a[j], acc.a[j]);
          acc.b[j] = fma2(d.b[j], x.b[j], acc.b[j]);
          d.a[j] = mul2(fma2(x.a[j], less2, mul2(d.a[j], g.a[j])), r2);
          d.b[j] = mul2(fma2(x.b[j], less2, mul2(d.b[j], g.b[j])), r2);
        }
        if (unit != 1.0f) scale_pairs(d, unit);  // (r of the head as it is may be no fp32 number)
        float fa[8], fb[8];
        runs_of<kInterleaved>(d, fa, fb);
        *reinterpret_cast<uint4*>(dx + h.a) = pack8(fa);
        *reinterpret_cast<uint4*>(dx + h.b) = pack8(fb);
      }
    }
    // this block's share of dg: its tokens one after the other
    __syncthreads();  // (the last share has been read)
    if (here.inside) {
      float* mine = sums + sub * dim;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const PairAt<kInterleaved> i(here, j);
        mine[i.first] = lo2(acc.a[j]), mine[i.first + i.step] = hi2(acc.a[j]);
        mine[i.second] = lo2(acc.b[j]), mine[i.second + i.step] = hi2(acc.b[j]);
      }
    }
    __syncthreads();
    const int share = kind ? units.shares_q + static_cast<int>(blockIdx.x) - units.first_k : static_cast<int>(blockIdx.x);
    for (int i = threadIdx.x; i < dim; i += kNormThreads) {
      float sum = 0.f;
      for (int t = 0; t < at_once; ++t) sum += sums[t * dim + i];
      p.partial[static_cast<int64_t>(share) * dim + i] = sum;
    }
  }
}

template <bool kInterleaved>
auto backward_kernel(int dim) {
  return dim == 64 ? norm_rope_backward_kernel<kInterleaved, 2> : dim == 128 ? norm_rope_backward_kernel<kInterleaved, 3>
         : dim == 256 ? norm_rope_backward_kernel<kInterleaved, 4> : norm_rope_backward_kernel<kInterleaved, -1>;
}

// dg of q and k from the blocks' shares, in their order: a block for 32 columns of one of them, a
// warp for every 32nd share, whose loads (19 of a full grid's 608 shares) are in flight together: 1 us less than
// eight at a time.
constexpr int kJoinColumns = 32, kJoinSlices = 32, kJoinBatch = 20;
__global__ void __launch_bounds__(kJoinColumns* kJoinSlices) norm_weight_kernel(const float* partial, int dim, int shares_q,
                                                                              int shares_k, float* dq_weight,
                                                                              float* dk_weight) {
  __shared__ float sums[kJoinSlices][kJoinColumns];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int col = blockIdx.x * kJoinColumns + lane, kind = blockIdx.y;
  const float* from = partial + (kind ? static_cast<int64_t>(shares_q) * dim : 0);
  const int n = kind ? shares_k : shares_q;
  float sum = 0.f;
  if (col < dim) {
    for (int i = slice; i < n; i += kJoinBatch * kJoinSlices) {
      float share[kJoinBatch];
#pragma unroll
      for (int j = 0; j < kJoinBatch; ++j) {
        const int at = i + j * kJoinSlices;
        share[j] = at < n ? __ldcg(from + static_cast<int64_t>(at) * dim + col) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kJoinBatch; ++j) sum += share[j];
    }
  }
  sums[slice][lane] = sum;
  __syncthreads();
  if (slice == 0 && col < dim) {
#pragma unroll
    for (int i = 1; i < kJoinSlices; ++i) sum += sums[i][lane];
    (kind ? dk_weight : dq_weight)[col] = sum;
  }
}

int lanes_log2_of(int dim) {
  int r = 0;
  while ((1 << r) < dim / 16) ++r;
  return r;
}

nvfp4_status launch_norm(NormJob p, int to, bool interleaved, cudaStream_t stream) {
  if (p.n_tokens == 0) return NVFP4_OK;
  p.lanes_log2 = lanes_log2_of(p.dim);
  p.inv_dim = 1.0f / static_cast<float>(p.dim);
  const int64_t threads = static_cast<int64_t>(p.n_tokens) << p.lanes_log2;
  const int total = p.heads[0] + p.heads[1] + p.heads[2];
  int per = 16;  // (as in rope.cu)
  while (per > 1 && threads * total / per < int64_t{152} * 1024) per /= 2;
  p.per_thread = per;
  int gy = 0;
  for (int i = 0; i < 3; ++i) gy += p.groups[i] = (p.heads[i] + per - 1) / per;
  if (gy > 65535) return NVFP4_ERR_SHAPE;
  const dim3 grid(static_cast<unsigned>((threads + kNormThreads - 1) / kNormThreads), gy);
  const auto kernel = to == kToRows ? (interleaved ? norm_rope_kernel<kToRows, true> : norm_rope_kernel<kToRows, false>)
                      : to == kToBf16 ? (interleaved ? norm_rope_kernel<kToBf16, true> : norm_rope_kernel<kToBf16, false>)
                                      : (interleaved ? norm_rope_kernel<kToE4M3, true> : norm_rope_kernel<kToE4M3, false>);
  if (launch_pdl(kernel, grid, dim3(kNormThreads), 0, stream, p) != cudaSuccess) return NVFP4_ERR_CUDA;
  return launched();
}

// The backward grid: as many blocks as the chip holds, or one for every four units where there are fewer.
BackwardUnits backward_units(int n_tokens, int n_heads, int n_kv_heads, int dim) {
  BackwardUnits b{};
  const int at_once = kNormThreads >> lanes_log2_of(dim);
  const int64_t steps = (n_tokens + at_once - 1) / at_once;
  b.of_q = steps * n_heads, b.all = steps * (n_heads + n_kv_heads);
  if (b.all == 0) return b;
  const int64_t most = 152 * 4, wanted = (b.all + 3) / 4, blocks = wanted < most ? wanted : most;
  b.per_block = static_cast<int>((b.all + blocks - 1) / blocks);
  b.blocks = static_cast<int>((b.all + b.per_block - 1) / b.per_block);
  b.shares_q = static_cast<int>((b.of_q + b.per_block - 1) / b.per_block);
  b.first_k = static_cast<int>(b.of_q / b.per_block);
  b.shares_k = n_kv_heads > 0 ? b.blocks - b.first_k : 0;
  return b;
}

nvfp4_status check_norm(const nvfp4_qk_norm* n, bool q, bool k) {
  if (!n || (q && !n->q_weight) || (k && !n->k_weight)) return NVFP4_ERR_NULL;
  if (n->weight_dtype != NVFP4_NORM_BF16 && n->weight_dtype != NVFP4_NORM_FP32) return NVFP4_ERR_LAYOUT;
  if (!std::isfinite(n->eps) || n->eps < 0.f) return NVFP4_ERR_SHAPE;
  const size_t size = n->weight_dtype == NVFP4_NORM_FP32 ? 4 : 2;
  if ((q && !aligned(n->q_weight, size)) || (k && !aligned(n->k_weight, size))) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

bool norm_sizes_ok(int n_tokens, int n_heads, int n_kv_heads, int head_dim) {
  return n_tokens >= 0 && n_heads >= 1 && n_kv_heads >= 0 && head_dim >= 16 && head_dim <= 512 && head_dim % 16 == 0 &&
         n_tokens < (1 << 30) && static_cast<int64_t>(n_heads) * head_dim < (1 << 30) &&
         static_cast<int64_t>(n_kv_heads) * head_dim < (1 << 30);
}

void set_norm(NormJob& p, const nvfp4_qk_norm* n) {
  p.weight[0] = n->q_weight, p.weight[1] = n->k_weight;
  p.weight_f32 = n->weight_dtype == NVFP4_NORM_FP32;
  p.eps = n->eps;
}

}  // namespace

nvfp4_status norm_error_word(uint32_t* v, int clear) { return unit_error_word(v, clear); }

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

nvfp4_status qk_norm_rope(const nvfp4_qk_norm* norm, const uint16_t* q, int64_t q_stride, int32_t n_heads,
                          const uint16_t* k, int64_t k_stride, int32_t n_kv_heads, int32_t n_tokens, int32_t head_dim,
                          const int32_t* positions, const double* inv_freq, int32_t rot_dim, float amplitude,
                          int32_t flags, uint16_t* q_out, int64_t q_out_stride, uint16_t* k_out, int64_t k_out_stride,
                          cudaStream_t stream) {
  const bool with_k = n_kv_heads > 0;
  if (const nvfp4_status st = check_norm(norm, true, with_k)) return st;
  if (n_tokens != 0 && (!q || !q_out || (with_k && (!k || !k_out)))) return NVFP4_ERR_NULL;
  if (!norm_sizes_ok(n_tokens, n_heads, n_kv_heads, head_dim)) return NVFP4_ERR_SHAPE;
  if (const nvfp4_status st = check_rows(q, q_stride, n_heads, head_dim)) return st;
  if (const nvfp4_status st = check_rows(q_out, q_out_stride, n_heads, head_dim)) return st;
  if (with_k) {
    if (const nvfp4_status st = check_rows(k, k_stride, n_kv_heads, head_dim)) return st;
    if (const nvfp4_status st = check_rows(k_out, k_out_stride, n_kv_heads, head_dim)) return st;
  }
  if (const nvfp4_status st = check_rotation(n_tokens, head_dim, positions, inv_freq, rot_dim, amplitude, flags,
                                             NVFP4_ROPE_INTERLEAVED))
    return st;
  NormJob p{};
  set_norm(p, norm);
  p.x[0] = q, p.x_stride[0] = q_stride, p.heads[0] = n_heads;
  p.x[1] = k, p.x_stride[1] = k_stride, p.heads[1] = n_kv_heads;
  p.y[0] = q_out, p.y_stride[0] = q_out_stride;
  p.y[1] = k_out, p.y_stride[1] = k_out_stride;
  p.positions = positions, p.inv_freq = inv_freq, p.amplitude = amplitude;
  p.n_tokens = n_tokens, p.dim = head_dim, p.rot = rot_dim;
  return launch_norm(p, kToRows, (flags & NVFP4_ROPE_INTERLEAVED) != 0, stream);
}

nvfp4_status kv_append_norm(const nvfp4_kv_cache* cache, const nvfp4_qk_norm* norm, const uint16_t* k, int64_t k_stride,
                            const uint16_t* v, int64_t v_stride, int32_t n_tokens, const int64_t* slots,
                            const int32_t* positions, const double* inv_freq, int32_t rot_dim, float amplitude,
                            int32_t flags, const uint16_t* q, int64_t q_stride, int32_t n_heads, uint16_t* q_out,
                            int64_t q_out_stride, cudaStream_t stream) {
  if (const nvfp4_status st = check_cache(cache)) return st;
  if (const nvfp4_status st = check_norm(norm, q != nullptr, true)) return st;
  if (n_tokens != 0 && (!k || !v || !slots || (q && !q_out) || (!q && q_out))) return NVFP4_ERR_NULL;
  if (!norm_sizes_ok(n_tokens, q ? n_heads : 1, cache->n_kv_heads, cache->head_dim)) return NVFP4_ERR_SHAPE;
  if (!aligned(slots, 8)) return NVFP4_ERR_ALIGN;
  if (const nvfp4_status st = check_rows(k, k_stride, cache->n_kv_heads, cache->head_dim)) return st;
  if (const nvfp4_status st = check_rows(v, v_stride, cache->n_kv_heads, cache->head_dim)) return st;
  if (q) {
    if (const nvfp4_status st = check_rows(q, q_stride, n_heads, cache->head_dim)) return st;
    if (const nvfp4_status st = check_rows(q_out, q_out_stride, n_heads, cache->head_dim)) return st;
  }
  if (const nvfp4_status st = check_rotation(n_tokens, cache->head_dim, positions, inv_freq, rot_dim, amplitude, flags,
                                             NVFP4_ROPE_INTERLEAVED))
    return st;
  NormJob p{};
  set_norm(p, norm);
  p.x[0] = q, p.x_stride[0] = q_stride, p.heads[0] = q ? n_heads : 0;
  p.x[1] = k, p.x_stride[1] = k_stride, p.heads[1] = cache->n_kv_heads;
  p.x[2] = v, p.x_stride[2] = v_stride, p.heads[2] = cache->n_kv_heads;
  p.y[0] = q_out, p.y_stride[0] = q_out_stride;
  p.cache[0] = static_cast<uint8_t*>(cache->k), p.cache[1] = static_cast<uint8_t*>(cache->v);
  p.scale[0] = cache->k_scale, p.scale[1] = cache->v_scale;
  p.page_stride = cache->page_stride, p.page_log2 = log2i(cache->page_size);
  p.n_slots = static_cast<int64_t>(cache->num_pages) * cache->page_size;
  p.slots = slots;
  p.positions = positions, p.inv_freq = inv_freq, p.amplitude = amplitude;
  p.n_tokens = n_tokens, p.dim = cache->head_dim, p.rot = rot_dim;
  return launch_norm(p, cache->dtype == NVFP4_KV_E4M3 ? kToE4M3 : kToBf16, (flags & NVFP4_ROPE_INTERLEAVED) != 0, stream);
}

size_t qk_norm_rope_workspace_bytes(int32_t n_tokens, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (!norm_sizes_ok(n_tokens, n_heads, n_kv_heads, head_dim)) return 0;
  const BackwardUnits b = backward_units(n_tokens, n_heads, n_kv_heads, head_dim);
  return (static_cast<size_t>(b.shares_q + b.shares_k) * head_dim + 4) * sizeof(float);
}

nvfp4_status qk_norm_rope_backward(const nvfp4_qk_norm* norm, const uint16_t* dq, int64_t dq_stride, const uint16_t* q,
                                   int64_t q_stride, int32_t n_heads, const uint16_t* dk, int64_t dk_stride,
                                   const uint16_t* k, int64_t k_stride, int32_t n_kv_heads, int32_t n_tokens,
                                   int32_t head_dim, const int32_t* positions, const double* inv_freq, int32_t rot_dim,
                                   float amplitude, int32_t flags, uint16_t* dq_out, int64_t dq_out_stride,
                                   uint16_t* dk_out, int64_t dk_out_stride, float* dq_weight, float* dk_weight, void* ws,
                                   size_t ws_bytes, cudaStream_t stream) {
  const bool with_k = n_kv_heads > 0;
  if (const nvfp4_status st = check_norm(norm, true, with_k)) return st;
  if (n_tokens != 0 && (!q || !dq || !dq_out || (with_k && (!k || !dk || !dk_out)))) return NVFP4_ERR_NULL;
  if (!dq_weight || (with_k && !dk_weight)) return NVFP4_ERR_NULL;
  if (!norm_sizes_ok(n_tokens, n_heads, n_kv_heads, head_dim)) return NVFP4_ERR_SHAPE;
  const struct {
    const void* x;
    int64_t stride;
    int heads;
  } rows[6] = {{q, q_stride, n_heads},     {dq, dq_stride, n_heads},    {dq_out, dq_out_stride, n_heads},
               {k, k_stride, n_kv_heads}, {dk, dk_stride, n_kv_heads}, {dk_out, dk_out_stride, n_kv_heads}};
  for (int i = 0; i < (with_k ? 6 : 3); ++i)
    if (const nvfp4_status st = check_rows(rows[i].x, rows[i].stride, rows[i].heads, head_dim)) return st;
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned(ws, 16)) return NVFP4_ERR_ALIGN;
  if (const nvfp4_status st = check_rotation(n_tokens, head_dim, positions, inv_freq, rot_dim, amplitude, flags,
                                             NVFP4_ROPE_INTERLEAVED))
    return st;
  if (!ws || ws_bytes < qk_norm_rope_workspace_bytes(n_tokens, n_heads, n_kv_heads, head_dim)) return NVFP4_ERR_WORKSPACE;
  const BackwardUnits b = backward_units(n_tokens, n_heads, n_kv_heads, head_dim);
  NormJob p{};
  set_norm(p, norm);
  p.x[0] = q, p.x_stride[0] = q_stride, p.heads[0] = n_heads;
  p.x[1] = k, p.x_stride[1] = k_stride, p.heads[1] = n_kv_heads;
  p.dy[0] = dq, p.dy_stride[0] = dq_stride, p.dy[1] = dk, p.dy_stride[1] = dk_stride;
  p.y[0] = dq_out, p.y_stride[0] = dq_out_stride, p.y[1] = dk_out, p.y_stride[1] = dk_out_stride;
  p.positions = positions, p.inv_freq = inv_freq, p.amplitude = amplitude;
  p.n_tokens = n_tokens, p.dim = head_dim, p.rot = rot_dim;
  p.lanes_log2 = lanes_log2_of(head_dim), p.inv_dim = 1.0f / static_cast<float>(head_dim);
  p.partial = static_cast<float*>(ws);
  // (without tokens there are no shares, and dg is zero)
  if (n_tokens > 0 &&
      launch_pdl((flags & NVFP4_ROPE_INTERLEAVED) ? backward_kernel<true>(head_dim) : backward_kernel<false>(head_dim),
                 dim3(b.blocks), dim3(kNormThreads), 0, stream, p, b) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  if (launch_pdl(norm_weight_kernel, dim3((head_dim + kJoinColumns - 1) / kJoinColumns, with_k ? 2 : 1),
                 dim3(kJoinColumns * kJoinSlices), 0, stream, static_cast<const float*>(p.partial), head_dim, b.shares_q,
                 b.shares_k, dq_weight, dk_weight) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  return launched();
}

}  // extern "C"
