// Launchers of the operators around the selection, one translation unit each;
// step_abi.cu has checked the arguments before it calls them.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "sparse_step.h"

namespace tki {

// Dynamic shared memory of one CTA that an SM grants.
constexpr int kMaxShared = 227 * 1024;

// Lets `kernel` take all of it, once per device.
template <auto kernel>
topk_status allow_shared(int dev) {
  static std::atomic<bool> done[64];
  if (done[dev].load(std::memory_order_relaxed)) return TOPK_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared) != cudaSuccess)
    return TOPK_ECUDA;
  done[dev].store(true, std::memory_order_relaxed);
  return TOPK_OK;
}

topk_status launch_rotary(const sparse_rotary_args& a, int sm_count, cudaStream_t stream);
topk_status launch_scores_bf16(const sparse_scores_args& a, int dev, int sm_count, cudaStream_t stream);
topk_status launch_scores_fp16(const sparse_scores_args& a, int dev, int sm_count, cudaStream_t stream);
topk_status launch_scores_e4m3(const sparse_scores_args& a, int dev, int sm_count, cudaStream_t stream);
topk_status launch_attention(const sparse_attention_args& a, int dev, int sm_count, cudaStream_t stream);

}  // namespace tki
