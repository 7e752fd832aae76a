// Indexer scores over a paged key cache (include/sparse_step.h,
// sparse_indexer_scores): the simple form, a thread per position.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "step_launch.cuh"

namespace tki {
namespace {

template <typename E>
__global__ void __launch_bounds__(128) scores_kernel(const sparse_scores_args a) {
  const int b = blockIdx.z, t = blockIdx.y;
  const int64_t s = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  const int64_t n = min(static_cast<int64_t>(a.lengths[static_cast<int64_t>(b) * a.T + t]), a.width);
  if (s >= n) return;
  const int32_t page = a.page_table[b * a.table_stride + s / a.page_size];
  float* out = a.out + b * a.out_seq_stride + t * a.out_token_stride + s;
  if (page < 0 || page >= a.num_pages) {
    *out = __int_as_float(0xff800000);
    return;
  }
  const int64_t place = s % a.page_size;
  const E* k = static_cast<const E*>(a.keys) + page * a.key_page_stride + place * a.key_token_stride;
  const E* q = static_cast<const E*>(a.q) + b * a.q_seq_stride + t * a.q_token_stride;
  const float* w = a.weights + (static_cast<int64_t>(b) * a.T + t) * a.H;
  float sum = 0.0f;
  for (int h = 0; h < a.H; ++h) {
    float dot = 0.0f;
    for (int d = 0; d < a.D; ++d) dot += static_cast<float>(q[h * a.q_head_stride + d]) * static_cast<float>(k[d]);
    sum += w[h] * (dot > 0.0f || dot != dot ? dot : 0.0f);
  }
  *out = a.key_scales != nullptr ? sum * a.key_scales[page * a.page_size + place] : sum;
}

}  // namespace

topk_status launch_scores(const sparse_scores_args& a, int, int, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.width + 127) / 128), a.T, a.B);
  if (a.T > 65535 || a.B > 65535) return TOPK_EINVAL;
  if (a.type == SPARSE_BF16) scores_kernel<__nv_bfloat16><<<grid, 128, 0, stream>>>(a);
  if (a.type == SPARSE_FP16) scores_kernel<__half><<<grid, 128, 0, stream>>>(a);
  if (a.type == SPARSE_E4M3) scores_kernel<__nv_fp8_e4m3><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? TOPK_OK : TOPK_ECUDA;
}

}  // namespace tki
