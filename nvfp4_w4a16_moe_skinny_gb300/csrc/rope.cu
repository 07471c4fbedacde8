// Rotary positions (rope_apply) and the append to a paged key/value cache with
// the rotation on the way (kv_append): one kernel over (token, head, chunk of 16
// values), bound by memory at prompt sizes and by the launch at decode sizes: 16,381 tokens of 32
// heads of 128 values (268 MB) take 46.0 us, 5.8 TB/s or 86% of the rate of a plain copy, 8,191 tokens
// quantized into a cache with their queries 33.0 us (82%); 16 tokens 2.9 us.
//
// The angle of pair i at position p is p * w_i radians.  In fp32 that product
// loses the angle at far positions (2^-24 of 131,072 radians is 0.008), so it is
// kept in turns as a 64-bit fraction: F = w / (2 pi) * 2^64 is an integer, p * F
// taken modulo 2^64 is the angle modulo a turn with no error but F's own
// rounding, and two integer multiplies replace an fp64 range reduction (the chip
// has few fp64 units).
#include <cmath>
#include <cstdint>

#include "launch.cuh"
#include "paged.cuh"

namespace nvfp4 {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kBatch = 2;  // heads whose loads a thread has in flight (a prompt's queries: 51 us with 1, 46 with 2, 47 with 4)

// What one launch does: up to three groups of heads per token (queries, keys,
// values), each read from rows and written to rows or to cache slots.
struct RopeJob {
  const uint16_t* x[3];      // rows of q, k, v (nullptr: none)
  int64_t x_stride[3];
  int heads[3];
  uint16_t* y;               // rotated queries
  int64_t y_stride;
  uint8_t* cache[2];         // pools of k and v
  const float* scale[2];     // E4M3 scales per kv head, or nullptr
  int64_t page_stride;       // elements
  int64_t n_slots;
  int page_log2;
  const int64_t* slots;
  const int32_t* positions;
  const double* inv_freq;
  float amplitude;
  int n_tokens, dim, rot;
  int interleaved, inverse;
  int per_thread;            // heads that one thread walks with the same angles
  int groups[3];             // ceil(heads / per_thread)
};

// w / (2 pi) as a 64-bit fraction of a turn (whole turns drop out), from the bits
// of w: M = w's significand in [2^63, 2^64), w = M * 2^(e - 63), and the high
// product of M with floor(2^66 / (2 pi)) is w / (2 pi) * 2^(65 - e).
__device__ __forceinline__ uint64_t turns_per_position(double w) {
  constexpr uint64_t kInvTwoPi = 0xA2F9836E4E441529ull;  // floor(2^66 / (2 pi)) = floor(2^65 / pi)
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(w));
  const int e = static_cast<int>((bits >> 52) & 0x7ff) - 1023;
  if (e < -64) return 0;  // below 2^-66 of a turn a position (zero and subnormals too)
  const uint64_t m = (bits << 11) | (1ull << 63);
  const uint64_t hi = __umul64hi(m, kInvTwoPi);
  const int s = 1 - e;
  if (s >= 64 || s <= -64) return 0;
  return s >= 0 ? hi >> s : hi << -s;
}

__device__ __forceinline__ void angle_of(const RopeJob& p, int pos, int pair, float& c, float& s) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns_per_position(__ldg(p.inv_freq + pair));
  // the nearest quarter turn is taken off as an integer, and the rest keeps all of its bits until it
  // becomes fp32, so that it has 24 of them near the axes too (a slow pair at position 1 turns by 2^-30)
  const uint32_t quarter = static_cast<uint32_t>((t + (1ull << 61)) >> 62);
  const int64_t rest = static_cast<int64_t>(t - (static_cast<uint64_t>(quarter) << 62));
  // |rest| from its halves: a conversion of 64 bits is longer (small calls 2.75 us against 2.65, the long prompt 46.3 against 46.0)
  const uint64_t size = rest < 0 ? -static_cast<uint64_t>(rest) : static_cast<uint64_t>(rest);
  const float half_turns = fmaf(__uint2float_rn(static_cast<uint32_t>(size >> 32)), 0x1p-31f,
                                __uint2float_rn(static_cast<uint32_t>(size)) * 0x1p-63f);
  float sr, cr;
  sincospif(rest < 0 ? -half_turns : half_turns, &sr, &cr);
  const bool swap = quarter & 1;
  const float cc = swap ? sr : cr, ss = swap ? cr : sr;
  c = (quarter == 1 || quarter == 2) ? -cc : cc;
  s = (quarter & 2) ? -ss : ss;
  c *= p.amplitude;
  s *= p.inverse ? -p.amplitude : p.amplitude;
}

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint4 v;
  v.x = f32x2_to_bf16x2(f[0], f[1]);
  v.y = f32x2_to_bf16x2(f[2], f[3]);
  v.z = f32x2_to_bf16x2(f[4], f[5]);
  v.w = f32x2_to_bf16x2(f[6], f[7]);
  return v;
}

// The reciprocal of a head's scale for products with values.  Those of scales near the ends of fp32 are not
// fp32's (the reciprocal of a subnormal is infinite, and zero times that NaN): there the scale, and
// with it the values, are first multiplied by `unit`, 2^64 or 2^-64.
struct HeadScale {
  float unit, inverse;
};
__device__ __forceinline__ HeadScale head_scale(float s) {
  const float unit = s < 0x1p-60f ? 0x1p64f : (s > 0x1p60f ? 0x1p-64f : 1.0f);
  return {unit, __frcp_rn(s * unit)};
}

// Eight values times the reciprocal of their head's scale as E4M3 codes, nearest-even, saturating at 448 (NaN
// stays NaN).  The reciprocal is rounded to fp32 once: a product is off by at most 2^-23 of the quotient, which
// moves a code only where the quotient is that near to the middle of two.  (For 8,191 tokens of 8 kv and 32 query
// heads a division a value took 36.3 us instead of 33.0, the rounded quotient by the product's remainder 34.2.)
__device__ __forceinline__ uint2 pack8_e4m3(float (&f)[8], const HeadScale s) {
  if (s.unit != 1.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= s.unit;
  }
  const float r = s.inverse;
  uint2 v;
  v.x = f32x2_to_e4m3x2(f[0] * r, f[1] * r) | f32x2_to_e4m3x2(f[2] * r, f[3] * r) << 16;
  v.y = f32x2_to_e4m3x2(f[4] * r, f[5] * r) | f32x2_to_e4m3x2(f[6] * r, f[7] * r) << 16;
  return v;
}

// One thread holds 16 values of a head: 8 pairs (two runs of 8 values half a
// rotation apart, or 16 adjacent ones where pairs interleave), or 16 values past
// the rotated part.  It computes its 8 angles once and walks `per_thread` heads
// with them; both runs are 16-byte loads, and the lanes of a token cover each
// head's row without gaps.  In place is safe: a thread writes what it read.
// (Registers for eight blocks an SM: small calls 2.85 us against 3.08 without the bound.)
template <bool kE4M3>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_kernel(const RopeJob p) {
  pdl_wait();
  pdl_launch_dependents();
  const int chunks = p.dim >> 4;
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int t = static_cast<int>(idx / chunks);
  const int chunk = static_cast<int>(idx - static_cast<int64_t>(t) * chunks);
  if (t >= p.n_tokens) return;
  int g = blockIdx.y, kind = 0;
  while (kind < 2 && g >= p.groups[kind]) g -= p.groups[kind++];
  const int h0 = g * p.per_thread, h1 = min(p.heads[kind], h0 + p.per_thread);
  const bool turn = kind < 2 && chunk < (p.rot >> 4);
  const bool split = turn && !p.interleaved;
  const int a = split ? 8 * chunk : 16 * chunk;           // first value of the two runs of 8
  const int b = split ? a + (p.rot >> 1) : a + 8;

  int64_t slot = 0;
  if (kind > 0) {
    slot = __ldg(p.slots + t);
    if (slot < 0) return;
    if (slot >= p.n_slots) {
      if (chunk == 0) atomicOr(&g_device_error, kErrPage);
      return;
    }
  }
  float c[8], s[8];
  if (turn) {
    const int pos = __ldg(p.positions + t);
#pragma unroll
    for (int i = 0; i < 8; ++i) angle_of(p, pos, 8 * chunk + i, c[i], s[i]);
  }
  const uint16_t* x = p.x[kind] + t * p.x_stride[kind];
  // element offset of (slot, head 0) in a pool, and from one head to the next
  const int64_t page = slot >> p.page_log2, off = slot & ((1 << p.page_log2) - 1);
  const int64_t base = kind ? page * p.page_stride + off * p.dim : t * p.y_stride;
  const int64_t head_step = kind ? static_cast<int64_t>(p.dim) << p.page_log2 : p.dim;
  // the loads of a batch of heads first: a store could alias a later load for all the compiler knows
  for (int hh = h0; hh < h1; hh += kBatch) {
    uint4 va[kBatch], vb[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = min(hh + k, h1 - 1);
      va[k] = *reinterpret_cast<const uint4*>(x + h * p.dim + a);
      vb[k] = *reinterpret_cast<const uint4*>(x + h * p.dim + b);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = hh + k;
      if (h >= h1) break;
      const int64_t o = base + h * head_step;
      uint16_t* y = kind ? reinterpret_cast<uint16_t*>(p.cache[kind - 1]) : p.y;
      if (!turn && !(kE4M3 && kind > 0)) {  // values that nothing turns are copied as they are
        *reinterpret_cast<uint4*>(y + o + a) = va[k];
        *reinterpret_cast<uint4*>(y + o + b) = vb[k];
        continue;
      }
      float fa[8], fb[8];
      unpack8(va[k], fa);
      unpack8(vb[k], fb);
      if (split) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = fa[i] * c[i] - fb[i] * s[i];
          fb[i] = fb[i] * c[i] + fa[i] * s[i];
          fa[i] = u;
        }
      } else if (turn) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = fa[2 * i] * c[i] - fa[2 * i + 1] * s[i];
          fa[2 * i + 1] = fa[2 * i + 1] * c[i] + fa[2 * i] * s[i];
          fa[2 * i] = u;
          const float w = fb[2 * i] * c[4 + i] - fb[2 * i + 1] * s[4 + i];
          fb[2 * i + 1] = fb[2 * i + 1] * c[4 + i] + fb[2 * i] * s[4 + i];
          fb[2 * i] = w;
        }
      }
      if (kE4M3 && kind > 0) {
        const HeadScale sc = head_scale(p.scale[kind - 1] ? __ldg(p.scale[kind - 1] + h) : 1.0f);
        *reinterpret_cast<uint2*>(p.cache[kind - 1] + o + a) = pack8_e4m3(fa, sc);
        *reinterpret_cast<uint2*>(p.cache[kind - 1] + o + b) = pack8_e4m3(fb, sc);
      } else {
        *reinterpret_cast<uint4*>(y + o + a) = pack8(fa);
        *reinterpret_cast<uint4*>(y + o + b) = pack8(fb);
      }
    }
  }
}

nvfp4_status launch_rope(RopeJob p, bool e4m3, cudaStream_t stream) {
  if (p.n_tokens == 0) return NVFP4_OK;
  // heads a thread walks: all of them reuse its angles, as long as the grid keeps
  // enough threads to fill the chip (the long prompt above: 116 us with one head a thread,
  // 48 with four, 46 with sixteen)
  const int64_t threads = static_cast<int64_t>(p.n_tokens) * (p.dim / 16);
  const int total = p.heads[0] + p.heads[1] + p.heads[2];
  int per = 16;
  while (per > 1 && threads * total / per < int64_t{152} * 1024) per /= 2;
  p.per_thread = per;
  int gy = 0;
  for (int i = 0; i < 3; ++i) gy += p.groups[i] = (p.heads[i] + per - 1) / per;
  if (gy > 65535) return NVFP4_ERR_SHAPE;
  const dim3 grid(static_cast<unsigned>((threads + kRopeThreads - 1) / kRopeThreads), gy);
  if (launch_pdl(e4m3 ? rope_kernel<true> : rope_kernel<false>, grid, dim3(kRopeThreads), 0, stream, p) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  return launched();
}

nvfp4_status check_rotation(int n_tokens, int dim, const int32_t* positions, const double* inv_freq, int rot,
                            float amplitude, int flags, int allowed) {
  if (flags & ~allowed) return NVFP4_ERR_SHAPE;
  if (rot < 0 || (rot % 16) || rot > dim || !std::isfinite(amplitude)) return NVFP4_ERR_SHAPE;
  if (rot > 0 && ((!positions && n_tokens != 0) || !inv_freq)) return NVFP4_ERR_NULL;
  if (rot > 0 && (!aligned(positions, 4) || !aligned(inv_freq, 8))) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

}  // namespace

nvfp4_status rope_error_word(uint32_t* v, int clear) { return unit_error_word(v, clear); }

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

nvfp4_status rope_frequencies(int32_t rot_dim, double theta, double factor, double trained_context, double slow,
                              double fast, double* inv_freq) {
  if (!inv_freq) return NVFP4_ERR_NULL;
  if (rot_dim < 16 || rot_dim > 512 || (rot_dim % 16)) return NVFP4_ERR_SHAPE;
  if (!std::isfinite(theta) || !std::isfinite(factor) || !std::isfinite(trained_context) || theta <= 1.0 ||
      factor < 1.0 || trained_context < 0.0)
    return NVFP4_ERR_SHAPE;
  if (trained_context > 0.0 && (!std::isfinite(slow) || !std::isfinite(fast) || fast <= slow)) return NVFP4_ERR_SHAPE;
  const double two_pi = 6.283185307179586476925286766559;
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double w = std::pow(theta, -2.0 * i / rot_dim);
    double keep = 0.0;
    if (trained_context > 0.0) {
      const double g = (trained_context * w / two_pi - slow) / (fast - slow);
      keep = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
    }
    inv_freq[i] = w * (keep + (1.0 - keep) / factor);
  }
  return NVFP4_OK;
}

nvfp4_status rope_apply(const uint16_t* x, int64_t x_stride, int32_t n_tokens, int32_t n_heads, int32_t head_dim,
                        const int32_t* positions, const double* inv_freq, int32_t rot_dim, float amplitude,
                        int32_t flags, uint16_t* y, int64_t y_stride, cudaStream_t stream) {
  if (n_tokens != 0 && (!x || !y)) return NVFP4_ERR_NULL;
  if (n_tokens < 0 || n_heads < 1 || head_dim < 16 || head_dim > 512 || (head_dim % 16) || rot_dim < 16)
    return NVFP4_ERR_SHAPE;
  if (const nvfp4_status st = check_rows(x, x_stride, n_heads, head_dim)) return st;
  if (const nvfp4_status st = check_rows(y, y_stride, n_heads, head_dim)) return st;
  if (const nvfp4_status st = check_rotation(n_tokens, head_dim, positions, inv_freq, rot_dim, amplitude, flags,
                                             NVFP4_ROPE_INTERLEAVED | NVFP4_ROPE_INVERSE))
    return st;
  RopeJob p{};
  p.x[0] = x, p.x_stride[0] = x_stride, p.heads[0] = n_heads;
  p.y = y, p.y_stride = y_stride;
  p.positions = positions, p.inv_freq = inv_freq, p.amplitude = amplitude;
  p.n_tokens = n_tokens, p.dim = head_dim, p.rot = rot_dim;
  p.interleaved = (flags & NVFP4_ROPE_INTERLEAVED) != 0, p.inverse = (flags & NVFP4_ROPE_INVERSE) != 0;
  return launch_rope(p, false, stream);
}

nvfp4_status kv_append(const nvfp4_kv_cache* cache, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                       int64_t v_stride, int32_t n_tokens, const int64_t* slots, const int32_t* positions,
                       const double* inv_freq, int32_t rot_dim, float amplitude, int32_t flags, const uint16_t* q,
                       int64_t q_stride, int32_t n_heads, uint16_t* q_out, int64_t q_out_stride, cudaStream_t stream) {
  if (const nvfp4_status st = check_cache(cache)) return st;
  if (n_tokens != 0 && (!k || !v || !slots || (q && !q_out) || (!q && q_out))) return NVFP4_ERR_NULL;
  if (n_tokens < 0 || (q && n_heads < 1)) return NVFP4_ERR_SHAPE;
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
  RopeJob p{};
  p.x[0] = q, p.x_stride[0] = q_stride, p.heads[0] = q ? n_heads : 0;
  p.x[1] = k, p.x_stride[1] = k_stride, p.heads[1] = cache->n_kv_heads;
  p.x[2] = v, p.x_stride[2] = v_stride, p.heads[2] = cache->n_kv_heads;
  p.y = q_out, p.y_stride = q_out_stride;
  p.cache[0] = static_cast<uint8_t*>(cache->k), p.cache[1] = static_cast<uint8_t*>(cache->v);
  p.scale[0] = cache->k_scale, p.scale[1] = cache->v_scale;
  p.page_stride = cache->page_stride, p.page_log2 = log2i(cache->page_size);
  p.n_slots = static_cast<int64_t>(cache->num_pages) * cache->page_size;
  p.slots = slots;
  p.positions = positions, p.inv_freq = inv_freq, p.amplitude = amplitude;
  p.n_tokens = n_tokens, p.dim = cache->head_dim, p.rot = rot_dim;
  p.interleaved = (flags & NVFP4_ROPE_INTERLEAVED) != 0;
  return launch_rope(p, cache->dtype == NVFP4_KV_E4M3, stream);
}

}  // extern "C"
