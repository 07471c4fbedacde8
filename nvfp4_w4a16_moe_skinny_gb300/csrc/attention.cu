// paged_attention: argument checks, tensor maps of the cache, dispatch.
#include <algorithm>
#include <cmath>

#include "attention.cuh"

namespace nvfp4 {
namespace {

// Tensor map of one pool, [num_pages, n_kv_heads, page_size, head_dim], whose rows are
// seen as blocks of 128 bytes (or one shorter block): boxes of one head's `box_rows`
// consecutive keys by one block, or by all blocks of the row.  Swizzled, so that eight
// rows of a 16-byte column fall into eight different groups of banks.
bool encode_pool_map(CUtensorMap* map, const nvfp4_kv_cache* c, void* base, int box_rows, bool whole_rows) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const bool fp8 = c->dtype == NVFP4_KV_E4M3;
  const cuuint64_t el = fp8 ? 1 : 2, row = c->head_dim * el, block = std::min<cuuint64_t>(128, row);
  const cuuint64_t dims[5] = {block / el, static_cast<cuuint64_t>(c->page_size), row / block,
                              static_cast<cuuint64_t>(c->n_kv_heads), static_cast<cuuint64_t>(c->num_pages)};
  const cuuint64_t strides[4] = {row, block, static_cast<cuuint64_t>(c->page_size) * row,
                                 static_cast<cuuint64_t>(c->page_stride) * el};
  const cuuint32_t box[5] = {static_cast<cuuint32_t>(block / el), static_cast<cuuint32_t>(box_rows),
                             whole_rows ? static_cast<cuuint32_t>(row / block) : 1, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base, dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            block == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps of both pools for the kernel and tile of `s`.
bool encode_maps(KvMaps* maps, const nvfp4_kv_cache* c, const AttnShape& s) {
  const int box = std::min(c->page_size, s.box_keys);
  return encode_pool_map(&maps->k, c, c->k, box, !s.chunk) && encode_pool_map(&maps->v, c, c->v, box, !s.chunk);
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

nvfp4_status kv_cache_maps(const nvfp4_kv_cache* cache, void* maps) {
  static_assert(sizeof(KvMaps) * kMapPairs == NVFP4_KV_MAPS_BYTES && alignof(KvMaps) <= 128, "maps");
  if (const nvfp4_status st = check_cache(cache)) return st;
  if (!maps) return NVFP4_ERR_NULL;
  if (!aligned(maps, 128)) return NVFP4_ERR_ALIGN;
  KvMaps all[kMapPairs];
  for (int64_t rows : {16, 32, 64, 65}) {  // one row count of each kind
    const AttnShape s = attn_shape(cache->head_dim, cache->dtype == NVFP4_KV_E4M3, rows, 1);
    if (!encode_maps(&all[s.maps], cache, s)) return NVFP4_ERR_CUDA;
  }
  std::copy(all, all + kMapPairs, static_cast<KvMaps*>(maps));
  return NVFP4_OK;
}

size_t paged_attention_workspace_bytes(int32_t n_tokens, int32_t n_seqs, int32_t max_new, int32_t n_heads,
                                       int32_t n_kv_heads, int32_t head_dim) {
  if (!attn_rows_ok(n_tokens, n_seqs, max_new, n_heads, n_kv_heads, head_dim)) return 0;
  const AttnShape s = attn_shape(head_dim, false, packed_rows(n_tokens, max_new, n_heads, n_kv_heads),
                                 static_cast<int64_t>(n_seqs) * n_kv_heads);
  const int grid = kAttnGrid * (s.chunk ? 1 : attn_ctas(head_dim, false, s.rw));
  const size_t share = static_cast<size_t>(s.tile_rows) * (head_dim + 2);  // sums of a row tile, references and sums of weights
  return kAttnCounterBytes + kAttnSplitBytes + 2 * grid * share * sizeof(float);
}

nvfp4_status paged_attention(const nvfp4_kv_cache* cache, const nvfp4_batch* batch, const uint16_t* q,
                             int64_t q_stride, int32_t n_tokens, int32_t n_heads, float scale, float softcap,
                             int32_t window, uint16_t* out, int64_t out_stride, float* lse, void* ws, size_t ws_bytes,
                             cudaStream_t stream) {
  if (const nvfp4_status st = check_cache(cache)) return st;
  if (!batch || (n_tokens != 0 && (!q || !out)) || !batch->cu_tokens) return NVFP4_ERR_NULL;
  if (batch->n_seqs != 0 && (!batch->kv_len || !batch->page_table)) return NVFP4_ERR_NULL;
  const int kv = cache->n_kv_heads, dim = cache->head_dim;
  if (!attn_sizes_ok(n_tokens, batch->n_seqs, batch->max_new, n_heads, kv, dim, batch->max_pages, cache->page_size))
    return NVFP4_ERR_SHAPE;
  if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f || window < 0) return NVFP4_ERR_SHAPE;
  if (const nvfp4_status st = check_rows(q, q_stride, n_heads, dim)) return st;
  if (const nvfp4_status st = check_rows(out, out_stride, n_heads, dim)) return st;
  if (!aligned(batch->cu_tokens, 4) || !aligned(batch->kv_len, 4) || !aligned(batch->page_table, 4) ||
      !aligned(lse, 4) || !aligned(ws, 32))
    return NVFP4_ERR_ALIGN;
  if (!ws || ws_bytes < paged_attention_workspace_bytes(n_tokens, batch->n_seqs, batch->max_new, n_heads, kv, dim))
    return NVFP4_ERR_WORKSPACE;
  if (n_tokens == 0 || batch->n_seqs == 0 || batch->max_new == 0) return NVFP4_OK;

  AttnJob p{};
  p.cu = batch->cu_tokens, p.kv_len = batch->kv_len, p.table = batch->page_table;
  p.n_seqs = batch->n_seqs, p.max_pages = batch->max_pages, p.n_tokens = n_tokens;
  p.n_heads = n_heads, p.n_kv = kv, p.group = n_heads / kv, p.by_group = fast_div(n_heads / kv);
  p.page_log2 = log2i(cache->page_size), p.num_pages = cache->num_pages;
  p.q = q, p.q_stride = q_stride, p.out = out, p.out_stride = out_stride, p.lse = lse;
  p.v_pool = cache->v, p.page_stride = cache->page_stride;
  p.k_scale = cache->k_scale, p.v_scale = cache->v_scale;
  p.scale = scale, p.softcap = softcap;
  p.window = attn_window(window);
  p.counters = static_cast<unsigned*>(ws);
  p.split = reinterpret_cast<int4*>(static_cast<uint8_t*>(ws) + kAttnCounterBytes);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kAttnCounterBytes + kAttnSplitBytes);
  const bool fp8 = cache->dtype == NVFP4_KV_E4M3;
  const AttnShape s = attn_shape(dim, fp8, packed_rows(n_tokens, batch->max_new, n_heads, kv),
                                 static_cast<int64_t>(batch->n_seqs) * kv);
  KvMaps maps;
  if (cache->maps)
    maps = static_cast<const KvMaps*>(cache->maps)[s.maps];
  else if (!encode_maps(&maps, cache, s))
    return NVFP4_ERR_CUDA;
  if (dim == 64) return dispatch_attention<64>(p, maps, fp8, s, stream);
  if (dim == 128) return dispatch_attention<128>(p, maps, fp8, s, stream);
  return dispatch_attention<256>(p, maps, fp8, s, stream);
}

}  // extern "C"
