// Attention over a cache in 8 bits, queries in fp16.
#include "cache_attention.cuh"

namespace tki {

topk_status launch_cache_attention_fp16(const sparse_attention_e4m3_args& a, int dev, int sm_count, cudaStream_t stream) {
  return launch_cache_attention<__half>(a, dev, sm_count, stream);
}

}  // namespace tki
