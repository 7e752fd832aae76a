// Attention over the selected entries of a paged cache
// (include/sparse_step.h, sparse_attention): the simple form, a warp per row
// and head, one pass with the running maximum and sum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "step_launch.cuh"

namespace tki {
namespace {

template <typename E>
__global__ void __launch_bounds__(32) attention_kernel(const sparse_attention_args a) {
  const int64_t row = blockIdx.x / a.Hq;
  const int h = static_cast<int>(blockIdx.x % a.Hq), g = h / (a.Hq / a.Hkv), lane = threadIdx.x;
  const int64_t b = row / a.T, t = row % a.T;
  const E* q = static_cast<const E*>(a.q) + b * a.q_seq_stride + t * a.q_token_stride + h * a.q_head_stride;
  constexpr int kPer = SPARSE_ATTENTION_MAX_D / 32;
  float o[kPer] = {};
  float m = __int_as_float(0xff800000), l = 0.0f;
  const int64_t qpos = a.query_positions != nullptr ? a.query_positions[row] : INT32_MAX;
  const int64_t first = a.first != nullptr ? a.first[row] : 0;
  for (int j = 0; j < a.K; ++j) {
    const int64_t pos = a.indices[row * a.K + j];
    if (pos < 0 || pos < first || pos > qpos || a.page_size == 0) continue;
    int64_t page = pos / a.page_size;
    const int64_t place = pos % a.page_size;
    if (a.page_table != nullptr) {
      if (page >= a.table_width) continue;
      page = a.page_table[b * a.table_stride + page];
    }
    if (page < 0 || page >= a.num_pages) continue;
    const E* k = static_cast<const E*>(a.k) + page * a.k_page_stride + place * a.k_token_stride + g * a.k_head_stride;
    const E* v = static_cast<const E*>(a.v) + page * a.v_page_stride + place * a.v_token_stride + g * a.v_head_stride;
    float z = 0.0f;
    for (int d = lane; d < a.D; d += 32) z += static_cast<float>(q[d]) * static_cast<float>(k[d]);
    for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
    z *= a.scale;
    if (a.softcap > 0.0f) z = a.softcap * tanhf(z / a.softcap);
    if (a.slopes != nullptr) z += a.slopes[h] * static_cast<float>(pos - qpos);
    const float top = fmaxf(m, z);
    const float base = top == __int_as_float(0xff800000) ? 0.0f : top;
    const float old = expf(m - base), p = expf(z - base);
    m = top;
    l = l * old + p;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < a.Dv) o[i] = o[i] * old + p * static_cast<float>(v[lane + 32 * i]);
  }
  E* out = static_cast<E*>(a.out) + (row * a.Hq + h) * a.Dv;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < a.Dv) out[lane + 32 * i] = static_cast<E>(l == 0.0f ? 0.0f : o[i] / l);
  if (a.lse != nullptr && lane == 0) a.lse[row * a.Hq + h] = l == 0.0f ? __int_as_float(0xff800000) : logf(l) + m;
}

}  // namespace

topk_status launch_attention(const sparse_attention_args& a, int, int, cudaStream_t stream) {
  const int64_t grid = static_cast<int64_t>(a.B) * a.T * a.Hq;
  if (grid > INT32_MAX) return TOPK_EINVAL;
  if (a.type == SPARSE_BF16) attention_kernel<__nv_bfloat16><<<static_cast<unsigned>(grid), 32, 0, stream>>>(a);
  if (a.type == SPARSE_FP16) attention_kernel<__half><<<static_cast<unsigned>(grid), 32, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? TOPK_OK : TOPK_ECUDA;
}

}  // namespace tki
