// What the kernels that turn heads share (rope.cu, head_norm.cu): angles, conversions of runs of
// eight values, the host-side checks of a rotation.
//
// The angle of pair i at position p is p * w_i radians.  In fp32 that product
// loses the angle at far positions (2^-24 of 131,072 radians is 0.008), so it is
// kept in turns as a 64-bit fraction: F = w / (2 pi) * 2^64 is an integer, p * F
// taken modulo 2^64 is the angle modulo a turn with no error but F's own
// rounding, and two integer multiplies replace an fp64 range reduction (the chip
// has few fp64 units).
#pragma once

#include <cmath>
#include <cstdint>

#include "launch.cuh"
#include "paged.cuh"

namespace nvfp4 {

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

// cos and sin of a pair's angle at a position, times the amplitude (`inverse`: the angle turned round).
__device__ __forceinline__ void angle_of(const double* inv_freq, float amplitude, bool inverse, int pos, int pair, float& c,
                                         float& s) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns_per_position(__ldg(inv_freq + pair));
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
  c *= amplitude;
  s *= inverse ? -amplitude : amplitude;
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

inline nvfp4_status check_rotation(int n_tokens, int dim, const int32_t* positions, const double* inv_freq, int rot,
                            float amplitude, int flags, int allowed) {
  if (flags & ~allowed) return NVFP4_ERR_SHAPE;
  if (rot < 0 || (rot % 16) || rot > dim || !std::isfinite(amplitude)) return NVFP4_ERR_SHAPE;
  if (rot > 0 && ((!positions && n_tokens != 0) || !inv_freq)) return NVFP4_ERR_NULL;
  if (rot > 0 && (!aligned(positions, 4) || !aligned(inv_freq, 8))) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

}  // namespace nvfp4
