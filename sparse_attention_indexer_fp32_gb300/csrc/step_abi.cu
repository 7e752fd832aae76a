// C ABI of the operators around the selection: argument checks, then the
// launch. See include/sparse_step.h for the contract.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "sparse_step.h"
#include "step_launch.cuh"

namespace {

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool whole16(int64_t elements, int64_t size) { return (elements * size) % 16 == 0; }

int64_t size_of(int32_t type) { return type == SPARSE_FP32 ? 4 : type == SPARSE_E4M3 ? 1 : 2; }

// The stride of a dimension of one element, which nothing is reached by, is 0
// from here on, whatever the caller's: no rule on strides counts it.
template <typename... S>
void unused(int64_t extent, S&... strides) {
  if (extent == 1) ((strides = 0), ...);
}

constexpr int kMaxDevices = 64;

struct Device {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  bool supported = false;
  int sm_count = 0;
};
Device g_devices[kMaxDevices];

// The current device and its SM count, checked once per device for sm_103.
topk_status ready(int* dev, int* sm_count) {
  const topk_status st = tki::status_of(cudaGetDevice(dev));
  if (st != TOPK_OK) return st;
  if (*dev < 0 || *dev >= kMaxDevices) return TOPK_EDEVICE;
  Device& d = g_devices[*dev];
  std::call_once(d.once, [&]() {
    int major = 0, minor = 0;
    d.err = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev);
    if (d.err == cudaSuccess) d.err = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev);
    if (d.err == cudaSuccess) d.err = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, *dev);
    d.supported = major == 10 && minor == 3;
  });
  if (d.err != cudaSuccess) return tki::status_of(d.err);
  if (!d.supported) return TOPK_EDEVICE;
  *sm_count = d.sm_count;
  return TOPK_OK;
}

}  // namespace

extern "C" {

topk_status sparse_rotary(const sparse_rotary_args* args, topk_stream_t stream) {
  if (args == nullptr) return TOPK_EINVAL;
  sparse_rotary_args a = *args;
  if (a.T < 0 || a.H < 0 || a.H > SPARSE_ROTARY_MAX_H || a.D < 1 || a.D > SPARSE_ROTARY_MAX_D) return TOPK_EINVAL;
  if (a.rotated < 2 || a.rotated % 2 != 0 || a.offset < 0 || a.offset > a.D - a.rotated) return TOPK_EINVAL;
  if (a.type != SPARSE_BF16 && a.type != SPARSE_FP16 && a.type != SPARSE_FP32) return TOPK_EINVAL;
  if (a.layout != SPARSE_ROTARY_HALF && a.layout != SPARSE_ROTARY_INTERLEAVED) return TOPK_EINVAL;
  if (!std::isfinite(a.scale)) return TOPK_EINVAL;
  if (a.slots != nullptr && (a.num_pages < 0 || a.page_size < 0)) return TOPK_EINVAL;
  if (a.T == 0 || a.H == 0 || (a.slots != nullptr && (a.num_pages == 0 || a.page_size == 0))) return TOPK_OK;
  if (a.slots != nullptr && a.num_pages > INT64_MAX / a.page_size) return TOPK_EINVAL;
  if (a.x == nullptr || a.out == nullptr || a.positions == nullptr || a.frequencies == nullptr) return TOPK_EINVAL;
  if (a.slots == nullptr) {
    unused(a.T, a.x_token_stride, a.out_token_stride);
  } else {
    unused(a.T, a.x_token_stride);
    unused(a.page_size, a.out_token_stride);
    unused(a.num_pages, a.out_page_stride);
  }
  unused(a.H, a.x_head_stride, a.out_head_stride);
  const uintptr_t size = static_cast<uintptr_t>(size_of(a.type));
  if (!aligned(a.x, size) || !aligned(a.out, size) || !aligned(a.positions, a.positions_64 ? 8 : 4) ||
      !aligned(a.frequencies, 8) || !aligned(a.slots, 4))
    return TOPK_EINVAL;
  int dev = 0, sms = 0;
  const topk_status st = ready(&dev, &sms);
  if (st != TOPK_OK) return st;
  return tki::launch_rotary(a, sms, reinterpret_cast<cudaStream_t>(stream));
}

topk_status sparse_indexer_scores(const sparse_scores_args* args, topk_stream_t stream) {
  if (args == nullptr) return TOPK_EINVAL;
  sparse_scores_args a = *args;
  if (a.type != SPARSE_BF16 && a.type != SPARSE_FP16 && a.type != SPARSE_E4M3) return TOPK_EINVAL;
  const int64_t size = size_of(a.type);
  if (a.B < 0 || a.T < 0 || a.H < 1 || a.H > SPARSE_SCORES_MAX_H) return TOPK_EINVAL;
  if (a.D < 1 || a.D > SPARSE_SCORES_MAX_D || !whole16(a.D, size)) return TOPK_EINVAL;
  if (a.width < 0 || a.width > INT32_MAX || a.table_width < 0 || a.num_pages < 0 || a.page_size < 0) return TOPK_EINVAL;
  if (a.B == 0 || a.T == 0 || a.width == 0) return TOPK_OK;
  if (a.page_size < 1 || a.table_stride < 0) return TOPK_EINVAL;
  if (a.table_width < (a.width + a.page_size - 1) / a.page_size) return TOPK_EINVAL;
  if (a.q == nullptr || a.weights == nullptr || a.lengths == nullptr || a.page_table == nullptr || a.out == nullptr ||
      (a.keys == nullptr && a.num_pages > 0))
    return TOPK_EINVAL;
  unused(a.B, a.q_seq_stride, a.table_stride, a.out_seq_stride);
  unused(a.T, a.q_token_stride, a.out_token_stride);
  unused(a.H, a.q_head_stride);
  unused(a.num_pages, a.key_page_stride);
  unused(a.page_size, a.key_token_stride);
  if (!aligned(a.keys, 16) || !whole16(a.key_page_stride, size) || !whole16(a.key_token_stride, size)) return TOPK_EINVAL;
  if (!aligned(a.q, static_cast<uintptr_t>(size)) || !aligned(a.weights, 4) || !aligned(a.key_scales, 4) ||
      !aligned(a.lengths, 4) || !aligned(a.page_table, 4) || !aligned(a.out, 4))
    return TOPK_EINVAL;
  int dev = 0, sms = 0;
  const topk_status st = ready(&dev, &sms);
  if (st != TOPK_OK) return st;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  switch (a.type) {
    case SPARSE_BF16: return tki::launch_scores_bf16(a, dev, sms, cs);
    case SPARSE_FP16: return tki::launch_scores_fp16(a, dev, sms, cs);
    default: return tki::launch_scores_e4m3(a, dev, sms, cs);
  }
}

topk_status sparse_attention(const sparse_attention_args* args, topk_stream_t stream) {
  if (args == nullptr) return TOPK_EINVAL;
  sparse_attention_args a = *args;
  if (a.type != SPARSE_BF16 && a.type != SPARSE_FP16) return TOPK_EINVAL;
  if (a.B < 0 || a.T < 0 || a.Hkv < 1 || a.Hq < 0 || a.Hq % a.Hkv != 0 || a.K < 0) return TOPK_EINVAL;
  if (a.D < 8 || a.D > SPARSE_ATTENTION_MAX_D || a.D % 8 != 0) return TOPK_EINVAL;
  if (a.Dv < 8 || a.Dv > SPARSE_ATTENTION_MAX_D || a.Dv % 8 != 0) return TOPK_EINVAL;
  if (!std::isfinite(a.scale) || !std::isfinite(a.softcap) || a.softcap < 0.0f) return TOPK_EINVAL;
  if (a.num_pages < 0 || a.page_size < 0 || a.table_width < 0 || a.table_stride < 0) return TOPK_EINVAL;
  if (a.page_table == nullptr && (a.query_positions != nullptr || a.first != nullptr || a.slopes != nullptr))
    return TOPK_EINVAL;
  if (a.slopes != nullptr && a.query_positions == nullptr) return TOPK_EINVAL;
  if (a.B == 0 || a.T == 0 || a.Hq == 0) return TOPK_OK;
  if (a.page_size > 0 && a.num_pages > INT64_MAX / a.page_size) return TOPK_EINVAL;
  const int64_t rows = static_cast<int64_t>(a.B) * a.T, heads = a.Hq / a.Hkv;
  if (rows > INT32_MAX || rows * a.Hkv > INT32_MAX || rows * a.Hkv * ((heads + 127) / 128) > INT32_MAX) return TOPK_EINVAL;
  const bool entries = a.K > 0 && a.num_pages > 0 && a.page_size > 0;
  if (a.q == nullptr || a.out == nullptr || (a.K > 0 && a.indices == nullptr) ||
      (entries && (a.k == nullptr || a.v == nullptr)))
    return TOPK_EINVAL;
  unused(a.B, a.q_seq_stride, a.table_stride);
  unused(a.T, a.q_token_stride);
  unused(a.Hq, a.q_head_stride);
  unused(a.num_pages, a.k_page_stride, a.v_page_stride);
  unused(a.page_size, a.k_token_stride, a.v_token_stride);
  unused(a.Hkv, a.k_head_stride, a.v_head_stride);
  if (!aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.out, 16) || !aligned(a.q, 2)) return TOPK_EINVAL;
  for (const int64_t s : {a.k_page_stride, a.k_token_stride, a.k_head_stride, a.v_page_stride, a.v_token_stride,
                          a.v_head_stride})
    if (!whole16(s, 2)) return TOPK_EINVAL;
  if (!aligned(a.indices, 4) || !aligned(a.page_table, 4) || !aligned(a.query_positions, 4) || !aligned(a.first, 4) ||
      !aligned(a.slopes, 4) || !aligned(a.lse, 4))
    return TOPK_EINVAL;
  int dev = 0, sms = 0;
  const topk_status st = ready(&dev, &sms);
  if (st != TOPK_OK) return st;
  return tki::launch_attention(a, dev, sms, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
