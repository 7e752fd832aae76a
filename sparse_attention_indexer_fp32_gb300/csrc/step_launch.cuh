// Launchers of the operators around the selection, one translation unit each;
// step_abi.cu has checked the arguments before it calls them.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "sparse_step.h"

namespace tki {

// Dynamic shared memory of one CTA that an SM grants.
constexpr int kMaxShared = 227 * 1024;

// The status of a CUDA call, by its own answer: the last error may be an
// earlier call's. What failed here is not left behind as the last error either.
inline topk_status status_of(cudaError_t err) {
  if (err == cudaSuccess) return TOPK_OK;
  (void)cudaGetLastError();
  return TOPK_ECUDA;
}

// Launches `kernel` on CTAs of `threads`, with `shared` bytes each.
template <typename P>
topk_status launch(void (*kernel)(P), const P& p, dim3 grid, int threads, size_t shared, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  return status_of(cudaLaunchKernelEx(&cfg, kernel, p));
}

// Lets `kernel` take all of it, once per device.
template <auto kernel>
topk_status allow_shared(int dev) {
  static std::atomic<bool> done[64];
  if (done[dev].load(std::memory_order_relaxed)) return TOPK_OK;
  const topk_status st = status_of(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared));
  if (st != TOPK_OK) return st;
  done[dev].store(true, std::memory_order_relaxed);
  return TOPK_OK;
}

topk_status launch_rotary(const sparse_rotary_args& a, int sm_count, cudaStream_t stream);
topk_status launch_scores_bf16(const sparse_scores_args& a, int dev, int sm_count, cudaStream_t stream);
topk_status launch_scores_fp16(const sparse_scores_args& a, int dev, int sm_count, cudaStream_t stream);
topk_status launch_scores_e4m3(const sparse_scores_args& a, int dev, int sm_count, cudaStream_t stream);
topk_status launch_attention(const sparse_attention_args& a, int dev, int sm_count, cudaStream_t stream);

}  // namespace tki
