// Checks of arguments and of the device that the C entry points share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "sparse_step.h"
#include "step_launch.cuh"

namespace tki {

inline bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline bool whole16(int64_t elements, int64_t size) { return (elements * size) % 16 == 0; }

inline int64_t size_of(int32_t type) { return type == SPARSE_FP32 ? 4 : type == SPARSE_E4M3 ? 1 : 2; }

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
inline Device g_devices[kMaxDevices];

// The current device and its SM count, checked once per device for sm_103.
inline topk_status ready(int* dev, int* sm_count) {
  const topk_status st = status_of(cudaGetDevice(dev));
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
  if (d.err != cudaSuccess) return status_of(d.err);
  if (!d.supported) return TOPK_EDEVICE;
  *sm_count = d.sm_count;
  return TOPK_OK;
}

}  // namespace tki
