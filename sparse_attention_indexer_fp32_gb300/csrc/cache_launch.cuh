// Launchers of the operators of a cache in 8 bits; cache_abi.cu has checked the
// arguments before it calls them.
#pragma once

#include <cuda_runtime.h>

#include "sparse_cache.h"

namespace tki {

topk_status launch_append(const sparse_append_args& a, int sm_count, cudaStream_t stream);
topk_status launch_cache_attention_bf16(const sparse_attention_e4m3_args& a, int dev, int sm_count, cudaStream_t stream);
topk_status launch_cache_attention_fp16(const sparse_attention_e4m3_args& a, int dev, int sm_count, cudaStream_t stream);

}  // namespace tki
