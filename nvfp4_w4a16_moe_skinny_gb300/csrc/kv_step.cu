// A step's bookkeeping on the GPU: page tables, slots, positions and ancestor masks from the
// requests' lengths (kv_assign), and an accepted path's cache rows moved next to each
// other (kv_accept).
#include <cstdint>

#include "launch.cuh"
#include "paged.cuh"

namespace nvfp4 {
namespace {

constexpr unsigned kErrStep = 8u;  // (g_device_error bit 3) pages, table columns or rows ran out; not a tree or path

constexpr int kAssignThreads = 1024, kAssignCtas = 8, kMostSeqs = 16384;

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

// Inclusive scan (sums held at 2^30) over the block; `all` gets the total.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = add_sat(v, u);
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int before = 0;
  all = 0;
  for (int w = 0; w < kAssignThreads / 32; ++w) {
    if (w == warp) before = all;
    all = add_sat(all, warp_sums[w]);
  }
  return add_sat(v, before);
}

// What a request asks for: its committed length, new tokens (clipped to the step's rows),
// pages held, pages to take and to give back.
struct Ask {
  int ctx, n, held, take, back;
};

__device__ __forceinline__ Ask ask_of(const AssignJob& p, int b, int start) {
  Ask a;
  const int fresh = __ldcg(p.fresh + b);
  a.ctx = fresh < 0 ? 0 : min(max(__ldcg(p.kv_len + b), 0), 1 << 30);
  a.held = min(max(__ldcg(p.held + b), 0), p.max_pages);
  a.n = min(max(fresh, 0), p.n_tokens - start);
  const int64_t end = static_cast<int64_t>(a.ctx) + a.n;
  const int need = static_cast<int>(min((end + (1 << p.page_log2) - 1) >> p.page_log2, static_cast<int64_t>(p.max_pages)));
  a.take = fresh < 0 ? 0 : max(0, need - a.held);
  a.back = fresh < 0 ? a.held : 0;
  return a;
}

// One cluster: every CTA scans the requests for itself and writes its share of the rows; nobody
// changes what another one reads (lengths, pages held, the free list) before all of them have read it.
__global__ void __cluster_dims__(kAssignCtas, 1, 1) __launch_bounds__(kAssignThreads) kv_assign_kernel(const AssignJob p) {
  extern __shared__ int smem[];
  int* const warp_sums = smem;                // [32]
  int* const start = smem + 32;               // [n_seqs + 1] first row of each request
  int* const first = start + p.n_seqs + 1;    // [n_seqs] its first page's place among those taken
  const int rank = static_cast<int>(blockIdx.x);
  pdl_wait();
  pdl_launch_dependents();
  unsigned bad = 0;
  int rows = 0, taken = 0, given = 0;
  for (int b0 = 0; b0 < p.n_seqs; b0 += kAssignThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    const int n = b < p.n_seqs ? min(max(__ldcg(p.fresh + b), 0), 1 << 30) : 0;
    int all;
    const int end = add_sat(rows, block_scan(n, warp_sums, all));
    if (b < p.n_seqs) {
      if (end > p.n_tokens) bad = kErrStep;
      start[b + 1] = min(end, p.n_tokens);
      if (b == 0) start[0] = 0;
    }
    rows = add_sat(rows, all);
  }
  rows = min(rows, p.n_tokens);
  __syncthreads();
  const int count = min(max(__ldcg(p.free_count), 0), p.num_free);
  for (int b0 = 0; b0 < p.n_seqs; b0 += kAssignThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    Ask a{};
    if (b < p.n_seqs) a = ask_of(p, b, start[b]);
    int all;
    const int end = add_sat(taken, block_scan(a.take, warp_sums, all));
    if (b < p.n_seqs) {
      first[b] = end - a.take;
      if (end > count || a.ctx + static_cast<int64_t>(a.n) > static_cast<int64_t>(p.max_pages) << p.page_log2) bad = kErrStep;
    }
    taken = add_sat(taken, all);
  }
  __syncthreads();
  const auto page_of = [&](int b, int held, int col) {  // -1: none
    if (col < held) return __ldcg(p.table + static_cast<int64_t>(b) * p.max_pages + col);
    const int at = count - 1 - (first[b] + col - held);
    return col < p.max_pages && at >= 0 ? __ldcg(p.free_pages + at) : -1;
  };
  // ---- rows
  for (int t = rank * kAssignThreads + static_cast<int>(threadIdx.x); t < p.n_tokens; t += kAssignCtas * kAssignThreads) {
    int64_t slot = -1;
    int position = 0;
    if (t < rows) {
      int lo = 0, hi = p.n_seqs - 1;  // the last request that starts at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const int b = lo, i = t - start[b];
      const int ctx = min(max(__ldcg(p.kv_len + b), 0), 1 << 30), held = min(max(__ldcg(p.held + b), 0), p.max_pages);
      const int at = ctx + i, page = page_of(b, held, at >> p.page_log2);
      if (page >= 0) slot = (static_cast<int64_t>(page) << p.page_log2) + (at & ((1 << p.page_log2) - 1));
      position = at;
      if (p.parents) {
        int depth = 0;
        for (int w = 0; w < p.words; ++w) {
          uint64_t mask = 0;
          for (int x = i; x >= 0;) {
            if (x >> 6 == w) mask |= 1ull << (x & 63);
            const int up = __ldg(p.parents + start[b] + x);
            if (up < -1 || up >= x) bad = kErrStep;
            x = up >= x ? -1 : up;
          }
          depth += __popcll(mask);
          p.masks[static_cast<int64_t>(t) * p.words + w] = static_cast<int64_t>(mask);
        }
        if (i >= 64 * p.words) bad = kErrStep;
        position = ctx + max(depth - 1, 0);
      }
    } else if (p.parents) {
      for (int w = 0; w < p.words; ++w) p.masks[static_cast<int64_t>(t) * p.words + w] = 0;
    }
    p.slots[t] = slot;
    p.positions[t] = position;
  }
  // ---- new entries of the page table, each CTA a share of the requests
  for (int b = rank * kAssignThreads + static_cast<int>(threadIdx.x); b < p.n_seqs; b += kAssignCtas * kAssignThreads) {
    const Ask a = ask_of(p, b, start[b]);
    for (int j = 0; j < a.take; ++j) {
      const int page = page_of(b, a.held, a.held + j);
      if (page < 0) break;
      p.table[static_cast<int64_t>(b) * p.max_pages + a.held + j] = page;
    }
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (bad) atomicOr(&g_device_error, bad);
  if (rank != 0) return;
  // ---- what the next step reads; finished requests' pages on top of the free list
  const int left = max(0, count - taken);
  for (int b0 = 0; b0 < p.n_seqs; b0 += kAssignThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    Ask a{};
    if (b < p.n_seqs) a = ask_of(p, b, start[b]);
    int all;
    const int end = add_sat(given, block_scan(a.back, warp_sums, all));
    if (b < p.n_seqs) {
      for (int j = 0; j < a.back; ++j) {
        const int64_t at = static_cast<int64_t>(left) + end - a.back + j;
        if (at < p.num_free) p.free_pages[at] = __ldcg(p.table + static_cast<int64_t>(b) * p.max_pages + j);
        else bad = kErrStep;
      }
      p.held[b] = a.held - a.back + max(0, min(a.take, count - first[b]));
      p.kv_len_out[b] = a.ctx + a.n;
      p.cu[b + 1] = start[b + 1];
      if (b == 0) p.cu[0] = 0;
    }
    given = add_sat(given, all);
  }
  if (threadIdx.x == 0) {
    *p.free_count = min(add_sat(left, given), p.num_free);
    if (p.n_seqs == 0) p.cu[0] = 0;
  }
  if (bad) atomicOr(&g_device_error, bad);
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
    if (threadIdx.x == 0) p.kv_len_out[b] = ctx + count;
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
  if (seqs < 0 || seqs > kMostSeqs || pages->max_pages < 1 || pages->num_free < 0 || rows < 0 || rows >= (1 << 30))
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
  p.masks = step->masks, p.n_tokens = rows, p.words = step->words;
  const size_t smem = (2 * static_cast<size_t>(seqs) + 33) * sizeof(int);
  if (set_smem(kv_assign_kernel, smem) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (launch_pdl(kv_assign_kernel, dim3(kAssignCtas), dim3(kAssignThreads), smem, stream, p) != cudaSuccess)
    return NVFP4_ERR_CUDA;
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
