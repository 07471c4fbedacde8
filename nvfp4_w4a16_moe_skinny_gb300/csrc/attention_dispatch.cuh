// Definitions behind dispatch_attention<kDim, kTree>, included by each attention_d<dim>.cu and
// attention_tree_d<dim>.cu translation unit, which instantiates them for its own only.
#pragma once

#include "attention_chunk.cuh"

namespace nvfp4 {

template <int kDim, bool kFp8, bool kTree>
nvfp4_status dispatch_rows(const AttnJob& p, const KvMaps& maps, const AttnShape& s, cudaStream_t stream) {
  if constexpr (kTree && kDim < 256)
    if (s.pair) return launch_attn_chunk<kDim, kFp8, kTree, true>(p, maps, stream);
  if (s.chunk) return launch_attn_chunk<kDim, kFp8, kTree, false>(p, maps, stream);
  if (s.rw == 1) return launch_attn_split<kDim, kFp8, 1, 4, kTree>(p, maps, stream);
  if (s.rw == 2) return launch_attn_split<kDim, kFp8, 2, 2, kTree>(p, maps, stream);
  return launch_attn_split<kDim, kFp8, 4, 1, kTree>(p, maps, stream);
}

template <int kDim, bool kTree>
nvfp4_status dispatch_attention(const AttnJob& p, const KvMaps& maps, bool fp8, const AttnShape& s,
                                cudaStream_t stream) {
  return fp8 ? dispatch_rows<kDim, true, kTree>(p, maps, s, stream) : dispatch_rows<kDim, false, kTree>(p, maps, s, stream);
}

template <int kDim, bool kTree>
nvfp4_status attention_error_word(uint32_t* v, int clear) {
  return unit_error_word(v, clear);
}

}  // namespace nvfp4
