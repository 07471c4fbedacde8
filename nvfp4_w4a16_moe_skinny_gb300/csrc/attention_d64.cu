// The attention kernels for heads of 64 values: one translation unit per head size
// so that they compile in parallel.
#include "attention_dispatch.cuh"

namespace nvfp4 {
template nvfp4_status dispatch_attention<64, false>(const AttnJob&, const KvMaps&, bool, const AttnShape&, cudaStream_t);
template nvfp4_status attention_error_word<64, false>(uint32_t*, int);
}  // namespace nvfp4
