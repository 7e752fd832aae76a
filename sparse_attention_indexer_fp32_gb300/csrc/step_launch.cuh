// Launchers of the operators around the selection, one translation unit each;
// step_abi.cu has checked the arguments before it calls them.
#pragma once

#include <cuda_runtime.h>

#include "sparse_step.h"

namespace tki {

// The current device's index and SM count; TOPK_EDEVICE unless it is sm_103.
topk_status current_device(int* dev, int* sm_count);

topk_status launch_rotary(const sparse_rotary_args& a, int sm_count, cudaStream_t stream);
topk_status launch_scores(const sparse_scores_args& a, int sm_count, cudaStream_t stream);
topk_status launch_attention(const sparse_attention_args& a, int sm_count, cudaStream_t stream);

}  // namespace tki
