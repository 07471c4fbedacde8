// A step's bookkeeping on the GPU: page tables, slots, positions and ancestor masks from the
// requests' lengths (kv_assign), and an accepted path's cache rows moved next to each
// other (kv_accept).
#include <cstdint>

#include "launch.cuh"
#include "paged.cuh"

namespace nvfp4 {
namespace {

constexpr unsigned kErrStep = 8u;  // (g_device_error bit 3) pages, table columns or rows ran out; not a tree or path

constexpr int kMostSeqs = 16384;
constexpr int kMostKept = 14336;  // requests whose lengths and pages fit into shared memory beside their places

struct AssignJob {
  int32_t* table;
  int32_t* held;
  int32_t* free_pages;
  int32_t* free_count;
  int n_seqs, max_pages, page_log2, num_free;
  const int32_t* kv_len;
  const int32_t* fresh;  // new tokens
  const int32_t* parents;
  int64_t* slots;
  int32_t* positions;
  int32_t* cu;
  int32_t* kv_len_out;
  int64_t* masks;
  int n_tokens, words;
};

// a + b for values of at most 2^30, held there
__device__ __forceinline__ int add_sat(int a, int b) { return min(static_cast<unsigned>(a) + static_cast<unsigned>(b), 1u << 30); }

// Inclusive scans (sums held at 2^30) of two values a thread over the block, and their totals.
template <int kThreads>
__device__ __forceinline__ void block_scan(int& x, int& y, int2* warp_sums, int& all_x, int& all_y) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x = add_sat(x, u), y = add_sat(y, v);
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = make_int2(x, y);
  __syncthreads();
  int2 w = lane < kWarps ? warp_sums[lane] : make_int2(0, 0);
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, w.x, o), v = __shfl_up_sync(0xffffffffu, w.y, o);
    if (lane >= o) w.x = add_sat(w.x, u), w.y = add_sat(w.y, v);
  }
  all_x = __shfl_sync(0xffffffffu, w.x, kWarps - 1), all_y = __shfl_sync(0xffffffffu, w.y, kWarps - 1);
  const int before_x = __shfl_sync(0xffffffffu, w.x, max(warp - 1, 0)), before_y = __shfl_sync(0xffffffffu, w.y, max(warp - 1, 0));
  if (warp > 0) x = add_sat(x, before_x), y = add_sat(y, before_y);
}

// What a request asks for: its committed length, new tokens, pages held, pages to take and to give back.
struct Ask {
  int ctx, n, held, take, back;
};

__device__ __forceinline__ Ask ask_of(const AssignJob& p, int b) {
  Ask a{};
  if (b >= p.n_seqs) return a;
  const int fresh = __ldcg(p.fresh + b), len = __ldcg(p.kv_len + b);
  a.held = min(max(__ldcg(p.held + b), 0), p.max_pages);
  a.ctx = fresh < 0 ? 0 : min(max(len, 0), 1 << 30);
  a.n = min(max(fresh, 0), 1 << 30);
  a.back = fresh < 0 ? a.held : 0;
  return a;
}

// Pages that a request takes for n new tokens.
__device__ __forceinline__ int pages_to_take(const AssignJob& p, const Ask& a, int n) {
  if (a.back > 0) return 0;
  const int64_t end = static_cast<int64_t>(a.ctx) + n;
  return max(0, static_cast<int>(min((end + (1 << p.page_log2) - 1) >> p.page_log2, static_cast<int64_t>(p.max_pages))) - a.held);
}

// Up to kFewRows rows of few requests: one CTA; else one cluster of eight, each of which scans the requests for itself
// and writes its share of the rows.  Nobody changes what another thread reads (lengths, pages held, the free list)
// before all of them have read it: that is the one barrier between the two halves, and why the launch is one
// cluster.  A step that finds its pages held already is bound by the launch and the chain of loads (requests, then page
// ids) and scans, and in trees by the walk up from each token: 16 requests of one token 2.8 us (3.8 in a cluster), trees of
// 164 tokens 3.7 (4.5), 421 rows of prompts 3.4 (3.8); trees of 665 tokens 6.8 in one CTA and 6.1, 1,821 rows of prompts 7.2
// and 4.0; 256 requests with 12,360 rows 4.9.
// Pages are taken, and given back, by one thread a request, one after the other, 0.21 us a page each way: 16 first tokens
// and their end 6.1 us for both calls, 256 prompts of 8,169 pages in all and their end 61, one prompt of 131,072 tokens in
// pages of 16 and its end 3.4 ms.  Each token walks up once for every four words of its mask: a chain of 256 tokens with its
// parents 17 us, of 4,096 15 ms (nine chains of 455 1.7 ms), without parents 3.8 and 38 us.
template <int kThreads, int kCtas>
__device__ __forceinline__ void assign_step(const AssignJob& p, int* smem) {
  int2* const warp_sums = reinterpret_cast<int2*>(smem);  // [32]
  int* const start = smem + 64;             // [n_seqs + 1] first row of each request
  int* const first = start + p.n_seqs + 1;  // [n_seqs] its first page's place among those taken
  int2* const kept = reinterpret_cast<int2*>(smem + 64 + 2 * p.n_seqs + 2);  // [n_seqs] committed length, pages held
  int* const own = reinterpret_cast<int*>(kept + p.n_seqs);  // parents of the CTA's rows (one CTA only)
  const bool keeps = kCtas == 1 || p.n_seqs <= kMostKept;
  const int rank = kCtas > 1 ? static_cast<int>(blockIdx.x) : 0, tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const Ask mine = ask_of(p, tid);
  const int count = min(max(__ldcg(p.free_count), 0), p.num_free);
  if (kCtas == 1 && p.parents)
    for (int t = tid; t < p.n_tokens; t += kThreads) own[t] = __ldg(p.parents + t);
  unsigned bad = 0;
  int rows = 0, taken = 0;
  bool gives = false;
  if (tid == 0) start[0] = 0;
  // rows and pages in one pass; again for the pages where the step's rows run out, as then requests get fewer of both
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int row0 = 0;
    taken = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.n_seqs; b0 += kThreads) {
      const int b = b0 + tid;
      const Ask a = b0 == 0 ? mine : ask_of(p, b);
      const int n = pass == 0 ? a.n : (b < p.n_seqs ? start[b + 1] - start[b] : 0);
      const int take = pages_to_take(p, a, n);
      int x = n, y = take, all_x, all_y;
      block_scan<kThreads>(x, y, warp_sums, all_x, all_y);
      if (b < p.n_seqs) {
        if (pass == 0 && keeps) kept[b] = make_int2(a.ctx, a.held);
        if (pass == 0) start[b + 1] = min(add_sat(row0, x), p.n_tokens);
        const int last = add_sat(taken, y);
        first[b] = last - take;
        if (last > count || (n > 0 && a.ctx + static_cast<int64_t>(n) > static_cast<int64_t>(p.max_pages) << p.page_log2))
          bad = kErrStep;
        gives = gives || a.back > 0;
      }
      row0 = add_sat(row0, all_x), taken = add_sat(taken, all_y);
    }
    if (pass == 0) rows = row0;
    __syncthreads();
    if (rows <= p.n_tokens) break;
    if (pass == 0) bad = 0;
    if (pass == 1) bad = kErrStep;
  }
  rows = min(rows, p.n_tokens);
  const auto page_of = [&](int b, int held, int col) {  // -1: none
    if (col < held) return __ldcg(p.table + static_cast<int64_t>(b) * p.max_pages + col);
    const int at = count - 1 - (first[b] + col - held);
    return col < p.max_pages && at >= 0 ? __ldcg(p.free_pages + at) : -1;
  };
  // ---- rows
  for (int t = rank * kThreads + tid; t < p.n_tokens; t += kCtas * kThreads) {
    int64_t slot = -1;
    int position = 0;
    if (t < rows) {
      int lo = 0, hi = p.n_seqs - 1;  // the last request that starts at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const int b = lo, row0 = start[b], i = t - row0;
      int2 r;
      if (keeps) {
        r = kept[b];
      } else {
        const Ask a = ask_of(p, b);
        r = make_int2(a.ctx, a.held);
      }
      const int ctx = r.x, at = ctx + i, page = page_of(b, r.y, at >> p.page_log2);
      if (page >= 0) slot = (static_cast<int64_t>(page) << p.page_log2) + (at & ((1 << p.page_log2) - 1));
      position = at;
      if (p.parents) {
        int depth = 0;
        for (int w0 = 0; w0 < p.words; w0 += 4) {  // four words of the mask at a walk up the tree
          uint64_t mask[4] = {};
          for (int x = i; x >= 0;) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (x >> 6 == w0 + k) mask[k] |= 1ull << (x & 63);
            const int up = kCtas == 1 ? own[row0 + x] : __ldg(p.parents + row0 + x);
            if (up < -1 || up >= x) bad = kErrStep;
            x = up >= x ? -1 : up;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (w0 + k < p.words) {
              depth += __popcll(mask[k]);
              p.masks[static_cast<int64_t>(t) * p.words + w0 + k] = static_cast<int64_t>(mask[k]);
            }
        }
        if (i >= 64 * p.words) bad = kErrStep;
        position = ctx + max(depth - 1, 0);
      } else if (p.masks) {  // a chain: the tokens up to this one
        for (int w = 0; w < p.words; ++w) {
          const int n = i + 1 - 64 * w;
          p.masks[static_cast<int64_t>(t) * p.words + w] = n >= 64 ? -1ll : (n > 0 ? (1ll << n) - 1 : 0ll);
        }
      }
    } else if (p.masks) {
      for (int w = 0; w < p.words; ++w) p.masks[static_cast<int64_t>(t) * p.words + w] = 0;
    }
    p.slots[t] = slot;
    p.positions[t] = position;
  }
  // ---- new entries of the page table, each CTA every eighth request of a block of them
#pragma unroll 1
  for (int b0 = 0; b0 < p.n_seqs; b0 += kThreads) {
    const int b = b0 + tid;
    if (b >= p.n_seqs || (kCtas > 1 && tid % kCtas != rank)) continue;
    const Ask a = b0 == 0 ? mine : ask_of(p, b);
    const int take = pages_to_take(p, a, start[b + 1] - start[b]);
    for (int j = 0; j < take; ++j) {
      const int page = page_of(b, a.held, a.held + j);
      if (page < 0) break;
      p.table[static_cast<int64_t>(b) * p.max_pages + a.held + j] = page;
    }
  }
  if (bad) atomicOr(&g_device_error, bad);
  if constexpr (kCtas > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank != 0) return;
    gives = __syncthreads_or(gives);
  } else {
    gives = __syncthreads_or(gives);
  }
  // ---- what the next step reads; finished requests' pages on top of the free list
  const int left = max(0, count - taken);
  int given = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.n_seqs; b0 += kThreads) {
    const int b = b0 + tid;
    const Ask a = b0 == 0 ? mine : ask_of(p, b);
    if (gives) {
      int x = a.back, none = 0, all, nothing;
      block_scan<kThreads>(x, none, warp_sums, all, nothing);
      const int from = add_sat(given, x) - a.back;
      for (int j = 0; j < a.back; ++j) {
        const int64_t at = static_cast<int64_t>(left) + from + j;
        if (at < p.num_free)
          p.free_pages[at] = __ldcg(p.table + static_cast<int64_t>(b) * p.max_pages + j);
        else
          atomicOr(&g_device_error, kErrStep);
      }
      given = add_sat(given, all);
    }
    if (b < p.n_seqs) {
      const int n = start[b + 1] - start[b];
      p.held[b] = a.held - a.back + max(0, min(pages_to_take(p, a, n), count - first[b]));
      p.kv_len_out[b] = a.ctx + n;
      p.cu[b + 1] = start[b + 1];
    }
  }
  if (tid == 0) {
    p.cu[0] = 0;
    *p.free_count = min(add_sat(left, given), p.num_free);
  }
}

constexpr int kFewThreads = 256, kFewRows = 512, kManyThreads = 1024, kManyCtas = 8;

__global__ void __launch_bounds__(kFewThreads) kv_assign_few_kernel(const AssignJob p) {
  __shared__ __align__(16) int smem[64 + 4 * kFewThreads + 2 + kFewRows];
  assign_step<kFewThreads, 1>(p, smem);
}

__global__ void __cluster_dims__(kManyCtas, 1, 1) __launch_bounds__(kManyThreads) kv_assign_kernel(const AssignJob p) {
  extern __shared__ __align__(16) int dynamic[];
  assign_step<kManyThreads, kManyCtas>(p, dynamic);
}

// ------------------------------------------------------------------ the accepted path

constexpr int kAcceptThreads = 128, kAcceptBatch = 8, kMostPath = 1024;

struct AcceptJob {
  uint8_t* pool[2];
  int64_t page_bytes, head_bytes;  // from one page to the next, from one head to the next
  int row_bytes, row_log2;         // of a key; its 16-byte chunks as a power of two
  int n_kv, page_log2, num_pages;
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* table;
  int n_seqs, max_pages;
  const int32_t* paths;
  int path_len;
  int32_t* kv_len_out;
};

// Byte offset of key `key` of head 0 in a pool, or -1 where its page is none.
__device__ __forceinline__ int64_t key_at(const AcceptJob& p, const int32_t* table, int key) {
  if (key < 0 || key >> p.page_log2 >= p.max_pages) return -1;
  const int page = __ldg(table + (key >> p.page_log2));
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) return -1;
  return page * p.page_bytes + static_cast<int64_t>(key & ((1 << p.page_log2) - 1)) * p.row_bytes;
}

// A block: one sequence and 128 16-byte columns of its K and V rows of all heads.  A path ascends, so
// path[d] >= d and a row is read before the path's own rows reach it: a thread moves its column of one
// entry after the other, kAcceptBatch loads in flight.
__global__ void __launch_bounds__(kAcceptThreads) kv_accept_kernel(const AcceptJob p) {
  __shared__ int64_t from[kMostPath], to[kMostPath];
  __shared__ int length;
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y;
  const int n = max(0, __ldg(p.cu + b + 1) - __ldg(p.cu + b)), len = __ldg(p.kv_len + b), ctx = len - n;
  const int32_t* path = p.paths + static_cast<int64_t>(b) * p.path_len;
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.max_pages;
  if (threadIdx.x == 0) length = p.path_len;
  __syncthreads();
  bool bad = false;
  for (int d = threadIdx.x; d < p.path_len; d += kAcceptThreads) {
    const int i = __ldg(path + d), before = d > 0 ? __ldg(path + d - 1) : -1;
    from[d] = to[d] = -1;
    const bool fits = i > before && i < n;
    if (!fits) {
      atomicMin(&length, d);
      continue;
    }
    if (i == d) continue;
    from[d] = key_at(p, table, ctx + i), to[d] = key_at(p, table, ctx + d);
  }
  __syncthreads();
  const int count = length;
  for (int d = threadIdx.x; d < count; d += kAcceptThreads)
    if (__ldg(path + d) != d && (from[d] < 0 || to[d] < 0) ) bad = true, from[d] = -1;
  if (threadIdx.x == 0 && count < p.path_len && __ldg(path + count) >= 0) bad = true;
  __syncthreads();
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) p.kv_len_out[b] = max(0, ctx + count);  // (kv_len may be below the new tokens)
    if (bad) atomicOr(&g_device_error, kErrStep);
  }
  const int columns = 2 * p.n_kv << p.row_log2, column = blockIdx.x * kAcceptThreads + threadIdx.x;
  if (column >= columns) return;
  const int row = column >> p.row_log2, head = row % p.n_kv;
  uint8_t* const at = p.pool[row / p.n_kv] + head * p.head_bytes + (column & ((1 << p.row_log2) - 1)) * 16;
  for (int d0 = 0; d0 < count; d0 += kAcceptBatch) {
    uint4 v[kAcceptBatch];
#pragma unroll
    for (int k = 0; k < kAcceptBatch; ++k)
      if (d0 + k < count && from[d0 + k] >= 0) v[k] = *reinterpret_cast<const uint4*>(at + from[d0 + k]);
#pragma unroll
    for (int k = 0; k < kAcceptBatch; ++k)
      if (d0 + k < count && from[d0 + k] >= 0) *reinterpret_cast<uint4*>(at + to[d0 + k]) = v[k];
  }
}

}  // namespace

nvfp4_status step_error_word(uint32_t* v, int clear) { return unit_error_word(v, clear); }

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

nvfp4_status kv_assign(const nvfp4_page_table* pages, const int32_t* kv_len, const int32_t* new_tokens,
                       const int32_t* parents, const nvfp4_step* step, cudaStream_t stream) {
  if (!pages || !step) return NVFP4_ERR_NULL;
  const int seqs = pages->n_seqs, rows = step->n_tokens;
  if (seqs < 0 || seqs > kMostSeqs || pages->max_pages < 1 || pages->num_free < 0 || pages->num_free >= (1 << 30) ||
      rows < 0 || rows >= (1 << 30))  // (sums of rows and pages are held at 2^30)
    return NVFP4_ERR_SHAPE;
  if (pages->page_size < 16 || pages->page_size > 256 || (pages->page_size & (pages->page_size - 1))) return NVFP4_ERR_SHAPE;
  if (static_cast<int64_t>(pages->max_pages) * pages->page_size >= (int64_t{1} << 30)) return NVFP4_ERR_SHAPE;
  if (step->words < 0 || step->words > 64 || (parents && step->words < 1)) return NVFP4_ERR_SHAPE;
  if (!pages->free_count || !step->cu_tokens || (pages->num_free > 0 && !pages->free_pages)) return NVFP4_ERR_NULL;
  if (seqs > 0 && (!pages->page_table || !pages->held || !kv_len || !new_tokens || !step->kv_len)) return NVFP4_ERR_NULL;
  if (rows > 0 && (!step->slots || !step->positions || (parents && !step->masks))) return NVFP4_ERR_NULL;
  for (const void* x : {static_cast<const void*>(pages->page_table), static_cast<const void*>(pages->held),
                        static_cast<const void*>(pages->free_pages), static_cast<const void*>(pages->free_count),
                        static_cast<const void*>(kv_len), static_cast<const void*>(new_tokens),
                        static_cast<const void*>(parents), static_cast<const void*>(step->positions),
                        static_cast<const void*>(step->cu_tokens), static_cast<const void*>(step->kv_len)})
    if (!aligned(x, 4)) return NVFP4_ERR_ALIGN;
  if (!aligned(step->slots, 8) || !aligned(step->masks, 8)) return NVFP4_ERR_ALIGN;
  AssignJob p{};
  p.table = pages->page_table, p.held = pages->held, p.free_pages = pages->free_pages, p.free_count = pages->free_count;
  p.n_seqs = seqs, p.max_pages = pages->max_pages, p.page_log2 = log2i(pages->page_size), p.num_free = pages->num_free;
  p.kv_len = kv_len, p.fresh = new_tokens, p.parents = rows > 0 ? parents : nullptr;
  p.slots = step->slots, p.positions = step->positions, p.cu = step->cu_tokens, p.kv_len_out = step->kv_len;
  p.masks = step->words > 0 ? step->masks : nullptr, p.n_tokens = rows, p.words = step->words;
  if (seqs <= kFewThreads && rows <= kFewRows) {
    if (launch_pdl(kv_assign_few_kernel, dim3(1), dim3(kFewThreads), 0, stream, p) != cudaSuccess) return NVFP4_ERR_CUDA;
    return launched();
  }
  const size_t smem = (static_cast<size_t>(seqs <= kMostKept ? 4 : 2) * seqs + 66) * sizeof(int);
  if (set_smem(kv_assign_kernel, smem) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (launch_pdl(kv_assign_kernel, dim3(kManyCtas), dim3(kManyThreads), smem, stream, p) != cudaSuccess) return NVFP4_ERR_CUDA;
  return launched();
}

nvfp4_status kv_accept(const nvfp4_kv_cache* cache, const nvfp4_batch* batch, const int32_t* paths, int32_t path_len,
                       int32_t* kv_len_out, cudaStream_t stream) {
  if (const nvfp4_status st = check_cache(cache)) return st;
  if (!batch) return NVFP4_ERR_NULL;
  const int seqs = batch->n_seqs;
  if (seqs < 0 || seqs > 65535 || path_len < 0 || path_len > kMostPath) return NVFP4_ERR_SHAPE;
  if (seqs == 0) return NVFP4_OK;
  if (!batch->cu_tokens || !batch->kv_len || !batch->page_table || !kv_len_out || (path_len > 0 && !paths))
    return NVFP4_ERR_NULL;
  if (batch->max_pages < 1 || static_cast<int64_t>(batch->max_pages) * cache->page_size >= (int64_t{1} << 30))
    return NVFP4_ERR_SHAPE;
  if (kv_len_out == batch->kv_len) return NVFP4_ERR_SHAPE;  // blocks of one sequence read it at their own times
  for (const void* x : {static_cast<const void*>(batch->cu_tokens), static_cast<const void*>(batch->kv_len),
                        static_cast<const void*>(batch->page_table), static_cast<const void*>(paths),
                        static_cast<const void*>(kv_len_out)})
    if (!aligned(x, 4)) return NVFP4_ERR_ALIGN;
  const int el = cache->dtype == NVFP4_KV_BF16 ? 2 : 1;
  AcceptJob p{};
  p.pool[0] = static_cast<uint8_t*>(cache->k), p.pool[1] = static_cast<uint8_t*>(cache->v);
  p.row_bytes = cache->head_dim * el, p.row_log2 = log2i(p.row_bytes / 16);
  p.page_bytes = cache->page_stride * el, p.head_bytes = static_cast<int64_t>(cache->page_size) * p.row_bytes;
  p.n_kv = cache->n_kv_heads, p.page_log2 = log2i(cache->page_size), p.num_pages = cache->num_pages;
  p.cu = batch->cu_tokens, p.kv_len = batch->kv_len, p.table = batch->page_table;
  p.n_seqs = seqs, p.max_pages = batch->max_pages;
  p.paths = paths, p.path_len = path_len, p.kv_len_out = kv_len_out;
  const int64_t columns = static_cast<int64_t>(2) * p.n_kv << p.row_log2;
  if (columns >= (1 << 30)) return NVFP4_ERR_SHAPE;
  const dim3 grid(static_cast<unsigned>((columns + kAcceptThreads - 1) / kAcceptThreads), seqs);
  if (launch_pdl(kv_accept_kernel, grid, dim3(kAcceptThreads), 0, stream, p) != cudaSuccess) return NVFP4_ERR_CUDA;
  return launched();
}

}  // extern "C"
