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
// A thread holds 16 values of a head as in rope.cu, 8 pairs, and walks heads with the same angles
// and weights; the lanes of a head share its sums by shuffles.
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

// The 16 values of a thread as 8 pairs: (a + i, b + i), or, where pairs interleave, (a + 2 i, a + 2 i + 1).
template <bool kInterleaved>
__device__ __forceinline__ void unpack_pairs(uint4 va, uint4 vb, float (&pa)[8], float (&pb)[8]) {
  float fa[8], fb[8];
  unpack8(va, fa);
  unpack8(vb, fb);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    pa[i] = kInterleaved ? (i < 4 ? fa[2 * i] : fb[2 * i - 8]) : fa[i];
    pb[i] = kInterleaved ? (i < 4 ? fa[2 * i + 1] : fb[2 * i - 7]) : fb[i];
  }
}
template <bool kInterleaved>
__device__ __forceinline__ void runs_of(const float (&pa)[8], const float (&pb)[8], float (&fa)[8], float (&fb)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    fa[i] = kInterleaved ? (i & 1 ? pb[i / 2] : pa[i / 2]) : pa[i];
    fb[i] = kInterleaved ? (i & 1 ? pb[4 + i / 2] : pa[4 + i / 2]) : pb[i];
  }
}

__device__ __forceinline__ float lanes_sum(float v, int lanes_log2) {
#pragma unroll
  for (int k = 0; k < 5; ++k)
    if (k < lanes_log2) v += __shfl_xor_sync(0xffffffffu, v, 1 << k);
  return v;
}

// A thread's own ring in shared memory, through which its loads of the next kAhead heads come without holding
// registers: 16-byte pieces, kParts a head, each read by the thread that copied it, so that no barrier is needed.
// A slot is filled again two heads after it was read.
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

// What a thread holds of its head: where its runs begin and whether its pairs turn.
struct Chunk {
  int token, chunk, a, b;
  bool inside, turn;
};

template <bool kInterleaved>
__device__ __forceinline__ Chunk chunk_at(const NormJob& p, int token, int chunk) {
  Chunk h;
  h.token = min(token, p.n_tokens - 1);
  h.chunk = chunk;
  h.inside = token < p.n_tokens && chunk < (p.dim >> 4);
  h.turn = chunk < (p.rot >> 4);
  const bool split = h.turn && !kInterleaved;
  h.a = split ? 8 * chunk : 16 * chunk;
  h.b = split ? h.a + (p.rot >> 1) : h.a + 8;
  if (chunk >= (p.dim >> 4)) h.a = h.b = 0;  // (a lane past the head: its copies are of nothing, from inside the row)
  return h;
}

template <bool kInterleaved>
__device__ __forceinline__ void load_weights(const NormJob& p, int kind, const Chunk& h, float (&ga)[8], float (&gb)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ia = kInterleaved ? h.a + 2 * i : h.a + i, ib = kInterleaved ? h.a + 2 * i + 1 : h.b + i;
    ga[i] = gb[i] = 0.f;
    if (!h.inside) continue;
    if (p.weight_f32) {
      ga[i] = __ldg(static_cast<const float*>(p.weight[kind]) + ia);
      gb[i] = __ldg(static_cast<const float*>(p.weight[kind]) + ib);
    } else {
      ga[i] = bf16_bits_to_f32(__ldg(static_cast<const uint16_t*>(p.weight[kind]) + ia));
      gb[i] = bf16_bits_to_f32(__ldg(static_cast<const uint16_t*>(p.weight[kind]) + ib));
    }
  }
}

enum { kToRows = 0, kToBf16 = 1, kToE4M3 = 2 };  // where keys and values go

template <int kTo, bool kInterleaved>
__global__ void __launch_bounds__(kNormThreads, 8) norm_rope_kernel(const NormJob p) {
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
    if (slot >= p.n_slots && live && h.chunk == 0) atomicOr(&g_device_error, kErrPage);
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
  float c[8], s[8], ga[8], gb[8];
  if (kind < 2) {
    load_weights<kInterleaved>(p, kind, h, ga, gb);
    if (h.turn) {
      const int pos = __ldg(p.positions + h.token);
#pragma unroll
      for (int i = 0; i < 8; ++i) angle_of(p.inv_freq, p.amplitude, false, pos, 8 * h.chunk + i, c[i], s[i]);
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
      float pa[8], pb[8];
      unpack_pairs<kInterleaved>(va, vb, pa, pb);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(pa[i], pa[i], fmaf(pb[i], pb[i], ss));
      ss = lanes_sum(ss, p.lanes_log2);
      float v = fmaf(ss, p.inv_dim, p.eps);
      const bool odd = out_of_range(v);
      if (__any_sync(0xffffffffu, odd)) {
        const float unit = odd ? scale_of(v) : 1.0f;
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          pa[i] *= unit, pb[i] *= unit;
          ss = fmaf(pa[i], pa[i], fmaf(pb[i], pb[i], ss));
        }
        v = fmaf(lanes_sum(ss, p.lanes_log2), p.inv_dim, p.eps * unit * unit);
      }
      const float r = rsqrtf(v);
      if (!live) continue;  // (the shuffles are done: the next head's are taken by all lanes again)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float na = pa[i] * r * ga[i], nb = pb[i] * r * gb[i];
        pa[i] = h.turn ? na * c[i] - nb * s[i] : na;
        pb[i] = h.turn ? nb * c[i] + na * s[i] : nb;
      }
      runs_of<kInterleaved>(pa, pb, fa, fb);
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

template <bool kInterleaved>
__global__ void __launch_bounds__(kNormThreads, 4) norm_rope_backward_kernel(const NormJob p) {
  __shared__ __align__(16) uint8_t ring_bytes[OwnRing<4>::kBytes];
  static_assert(sizeof(ring_bytes) >= kNormThreads * 16 * sizeof(float), "the sums at the end");
  float* const sums = reinterpret_cast<float*>(ring_bytes);  // [tokens of the block][dim], after the loop
  const OwnRing<4> ring{smem_addr(ring_bytes)};
  pdl_wait();
  pdl_launch_dependents();
  const int lanes = 1 << p.lanes_log2, at_once = kNormThreads >> p.lanes_log2;
  const int sub = threadIdx.x >> p.lanes_log2, chunk = threadIdx.x & (lanes - 1);
  const int g = static_cast<int>(blockIdx.y) - p.groups[0], kind = g >= 0 ? 1 : 0;
  const int h0 = (kind ? g : static_cast<int>(blockIdx.y)) * p.per_thread, h1 = min(p.heads[kind], h0 + p.per_thread);
  Chunk h = chunk_at<kInterleaved>(p, 0, chunk);
  float ga[8], gb[8], acc_a[8], acc_b[8];
  load_weights<kInterleaved>(p, kind, h, ga, gb);
#pragma unroll
  for (int i = 0; i < 8; ++i) acc_a[i] = acc_b[i] = 0.f;
  const int step = static_cast<int>(gridDim.x) * at_once, first = static_cast<int>(blockIdx.x) * at_once;
  // the copies run through the same tokens and heads, ahead of the loop
  int copied = 0, copy_t = first, copy_h = h0;
  const auto fetch = [&]() {
    if (copy_t < p.n_tokens) {
      const Chunk f = chunk_at<kInterleaved>(p, copy_t + sub, chunk);
      const uint16_t* x = p.x[kind] + f.token * p.x_stride[kind] + copy_h * p.dim;
      const uint16_t* dy = p.dy[kind] + f.token * p.dy_stride[kind] + copy_h * p.dim;
      const uint32_t bytes = f.inside ? 16 : 0;
      ring.copy(copied, 0, x + f.a, bytes);
      ring.copy(copied, 1, x + f.b, bytes);
      ring.copy(copied, 2, dy + f.a, bytes);
      ring.copy(copied, 3, dy + f.b, bytes);
      ++copied;
      if (++copy_h == h1) copy_h = h0, copy_t += step;
    }
    ring.commit();
  };
#pragma unroll
  for (int i = 0; i < ring.kAhead; ++i) fetch();
  int at = 0;
  for (int t0 = first; t0 < p.n_tokens; t0 += step) {
    h = chunk_at<kInterleaved>(p, t0 + sub, chunk);
    float c[8], s[8];
    if (h.turn) {
      const int pos = __ldg(p.positions + h.token);
#pragma unroll
      for (int i = 0; i < 8; ++i) angle_of(p.inv_freq, p.amplitude, false, pos, 8 * chunk + i, c[i], s[i]);
    }
    uint16_t* dx = p.y[kind] + h.token * p.y_stride[kind];
    for (int hh = h0; hh < h1; ++hh, ++at) {
      ring.arrived();
      const uint4 v[4] = {ring.read(at, 0), ring.read(at, 1), ring.read(at, 2), ring.read(at, 3)};
      fetch();
      float pa[8], pb[8], ua[8], ub[8];
      unpack_pairs<kInterleaved>(v[0], v[1], pa, pb);
      unpack_pairs<kInterleaved>(v[2], v[3], ua, ub);
      if (h.turn) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = ua[i] * c[i] + ub[i] * s[i];
          ub[i] = ub[i] * c[i] - ua[i] * s[i];
          ua[i] = u;
        }
      }
      float ss = 0.f, zx = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(pa[i], pa[i], fmaf(pb[i], pb[i], ss));
        zx = fmaf(ua[i] * ga[i], pa[i], fmaf(ub[i] * gb[i], pb[i], zx));
      }
      ss = lanes_sum(ss, p.lanes_log2);
      zx = lanes_sum(zx, p.lanes_log2);
      float var = fmaf(ss, p.inv_dim, p.eps), unit = 1.0f;
      const bool odd = out_of_range(var);
      if (__any_sync(0xffffffffu, odd)) {
        unit = odd ? scale_of(var) : 1.0f;
        ss = zx = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          pa[i] *= unit, pb[i] *= unit;
          ss = fmaf(pa[i], pa[i], fmaf(pb[i], pb[i], ss));
          zx = fmaf(ua[i] * ga[i], pa[i], fmaf(ub[i] * gb[i], pb[i], zx));
        }
        var = fmaf(lanes_sum(ss, p.lanes_log2), p.inv_dim, p.eps * unit * unit);
        zx = lanes_sum(zx, p.lanes_log2);
      }
      const float r = rsqrtf(var), along = zx * p.inv_dim * r, out = r * unit;
      if (!h.inside) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float na = pa[i] * r, nb = pb[i] * r;
        acc_a[i] = fmaf(ua[i], na, acc_a[i]);
        acc_b[i] = fmaf(ub[i], nb, acc_b[i]);
        ua[i] = out * (ua[i] * ga[i] - na * along);
        ub[i] = out * (ub[i] * gb[i] - nb * along);
      }
      float fa[8], fb[8];
      runs_of<kInterleaved>(ua, ub, fa, fb);
      *reinterpret_cast<uint4*>(dx + hh * p.dim + h.a) = pack8(fa);
      *reinterpret_cast<uint4*>(dx + hh * p.dim + h.b) = pack8(fb);
    }
  }
  // this block's share of dg: its tokens one after the other
  __syncthreads();  // (where the ring was)
  if (chunk < (p.dim >> 4)) {
    float* mine = sums + sub * p.dim;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mine[kInterleaved ? h.a + 2 * i : h.a + i] = acc_a[i];
      mine[kInterleaved ? h.a + 2 * i + 1 : h.b + i] = acc_b[i];
    }
  }
  __syncthreads();
  float* share = p.partial + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * p.dim;
  for (int i = threadIdx.x; i < p.dim; i += kNormThreads) {
    float sum = 0.f;
    for (int t = 0; t < at_once; ++t) sum += sums[t * p.dim + i];
    share[i] = sum;
  }
}

// dg of q and k from the blocks' shares, in their order: a block for 32 columns of one of them, a
// warp for every 32nd share.
constexpr int kJoinColumns = 32, kJoinSlices = 32;
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
#pragma unroll 8
    for (int i = slice; i < n; i += kJoinSlices) sum += __ldcg(from + static_cast<int64_t>(i) * dim + col);
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

// The backward grid: heads a thread walks, blocks over tokens and over heads.
struct BackwardPlan {
  int per_thread, groups[2], blocks;
  int shares() const { return (groups[0] + groups[1]) * blocks; }
};
BackwardPlan backward_plan(int n_tokens, int n_heads, int n_kv_heads, int dim) {
  BackwardPlan b;
  const int lanes_log2 = lanes_log2_of(dim);
  const int64_t threads = static_cast<int64_t>(n_tokens) << lanes_log2;
  b.per_thread = 8;
  while (b.per_thread > 1 && threads * (n_heads + n_kv_heads) / b.per_thread < int64_t{152} * 512) b.per_thread /= 2;
  b.groups[0] = (n_heads + b.per_thread - 1) / b.per_thread;
  b.groups[1] = (n_kv_heads + b.per_thread - 1) / b.per_thread;
  const int64_t all = (threads + kNormThreads - 1) / kNormThreads, fill = 152 * 4 / (b.groups[0] + b.groups[1]);
  b.blocks = static_cast<int>(all < fill ? all : (fill < 1 ? 1 : fill));
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
  const BackwardPlan b = backward_plan(n_tokens, n_heads, n_kv_heads, head_dim);
  return (static_cast<size_t>(b.shares()) * head_dim + 4) * sizeof(float);
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
  const BackwardPlan b = backward_plan(n_tokens, n_heads, n_kv_heads, head_dim);
  if (b.groups[0] + b.groups[1] > 65535) return NVFP4_ERR_SHAPE;
  NormJob p{};
  set_norm(p, norm);
  p.x[0] = q, p.x_stride[0] = q_stride, p.heads[0] = n_heads;
  p.x[1] = k, p.x_stride[1] = k_stride, p.heads[1] = n_kv_heads;
  p.dy[0] = dq, p.dy_stride[0] = dq_stride, p.dy[1] = dk, p.dy_stride[1] = dk_stride;
  p.y[0] = dq_out, p.y_stride[0] = dq_out_stride, p.y[1] = dk_out, p.y_stride[1] = dk_out_stride;
  p.positions = positions, p.inv_freq = inv_freq, p.amplitude = amplitude;
  p.n_tokens = n_tokens, p.dim = head_dim, p.rot = rot_dim;
  p.lanes_log2 = lanes_log2_of(head_dim), p.inv_dim = 1.0f / static_cast<float>(head_dim);
  p.per_thread = b.per_thread, p.groups[0] = b.groups[0], p.groups[1] = b.groups[1];
  p.partial = static_cast<float*>(ws);
  // (without tokens there are no shares, and dg is zero)
  if (n_tokens > 0 &&
      launch_pdl((flags & NVFP4_ROPE_INTERLEAVED) ? norm_rope_backward_kernel<true> : norm_rope_backward_kernel<false>,
                 dim3(b.blocks, b.groups[0] + b.groups[1]), dim3(kNormThreads), 0, stream, p) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  const int shares = n_tokens > 0 ? b.blocks : 0;
  if (launch_pdl(norm_weight_kernel, dim3((head_dim + kJoinColumns - 1) / kJoinColumns, with_k ? 2 : 1),
                 dim3(kJoinColumns * kJoinSlices), 0, stream, static_cast<const float*>(p.partial), head_dim,
                 b.groups[0] * shares, b.groups[1] * shares, dq_weight, dk_weight) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  return launched();
}

}  // extern "C"
