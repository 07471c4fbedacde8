// What the rotary, append and attention kernels share: the host-side checks of a
// paged cache and of rows of heads, and small conversions.
#pragma once

#include "common.cuh"

namespace nvfp4 {

constexpr unsigned kErrPage = 4u;  // a page id or slot outside its pool (g_device_error bit 2)

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int log2i(int v) {
  int r = 0;
  while ((1 << (r + 1)) <= v) ++r;
  return r;
}

// rows of `heads` heads of `dim` bf16 values, `stride` elements apart
inline nvfp4_status check_rows(const void* x, int64_t stride, int heads, int dim) {
  if (stride < static_cast<int64_t>(heads) * dim) return NVFP4_ERR_SHAPE;
  if (!aligned(x, 16) || (stride % 8)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

inline nvfp4_status check_cache(const nvfp4_kv_cache* c) {
  if (!c || !c->k || !c->v) return NVFP4_ERR_NULL;
  if (c->dtype != NVFP4_KV_BF16 && c->dtype != NVFP4_KV_E4M3) return NVFP4_ERR_LAYOUT;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return NVFP4_ERR_SHAPE;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return NVFP4_ERR_SHAPE;
  if (c->num_pages < 1 || c->n_kv_heads < 1) return NVFP4_ERR_SHAPE;
  if (c->page_stride < static_cast<int64_t>(c->n_kv_heads) * c->page_size * c->head_dim) return NVFP4_ERR_SHAPE;
  const int size = c->dtype == NVFP4_KV_BF16 ? 2 : 1;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || (c->page_stride * size) % 16) return NVFP4_ERR_ALIGN;
  if (c->dtype == NVFP4_KV_BF16 && (c->k_scale || c->v_scale)) return NVFP4_ERR_LAYOUT;
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || !aligned(c->maps, 128)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

// The device error word of the calling translation unit: read into *v, cleared if `clear`.
static nvfp4_status unit_error_word(uint32_t* v, int clear) {
  unsigned w = 0;
  if (cudaMemcpyFromSymbol(&w, g_device_error, sizeof(w)) != cudaSuccess) return NVFP4_ERR_CUDA;
  *v = w;
  if (clear) {
    const unsigned z = 0;
    if (cudaMemcpyToSymbol(g_device_error, &z, sizeof(z)) != cudaSuccess) return NVFP4_ERR_CUDA;
  }
  return NVFP4_OK;
}

// Two floats to a bf16x2 (lo in the low half), rounded to nearest even.
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two floats to E4M3 codes (lo in the low byte), nearest-even, saturating.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
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
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

}  // namespace nvfp4
