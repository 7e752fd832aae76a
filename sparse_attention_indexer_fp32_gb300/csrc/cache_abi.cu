// C ABI of the operators of a cache in 8 bits: argument checks, then the
// launch. See include/sparse_cache.h for the contract.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "cache_launch.cuh"
#include "sparse_cache.h"
#include "step_checks.cuh"

using namespace tki;

extern "C" {

topk_status sparse_append(const sparse_append_args* args, topk_stream_t stream) {
  if (args == nullptr) return TOPK_EINVAL;
  sparse_append_args a = *args;
  const bool values = a.v != nullptr, scaled = a.cache_type == SPARSE_E4M3;
  if (a.type != SPARSE_BF16 && a.type != SPARSE_FP16 && a.type != SPARSE_FP32) return TOPK_EINVAL;
  if (!scaled && a.cache_type != a.type) return TOPK_EINVAL;
  if (a.T < 0 || a.H < 0 || a.H > SPARSE_APPEND_MAX_H || a.D < 1 || a.D > SPARSE_APPEND_MAX_D) return TOPK_EINVAL;
  if (values && (a.Dv < 1 || a.Dv > SPARSE_APPEND_MAX_D)) return TOPK_EINVAL;
  if (a.rotated < 0 || a.rotated % 2 != 0 || a.offset < 0 || a.rotated > a.D || a.offset > a.D - a.rotated) return TOPK_EINVAL;
  if (a.layout != SPARSE_ROTARY_HALF && a.layout != SPARSE_ROTARY_INTERLEAVED) return TOPK_EINVAL;
  if (!std::isfinite(a.scale)) return TOPK_EINVAL;
  if (a.num_pages < 0 || a.page_size < 0) return TOPK_EINVAL;
  if (scaled && a.page_size > 0 && (a.blocks < 1 || a.page_size % a.blocks != 0)) return TOPK_EINVAL;
  if (a.T == 0 || a.H == 0 || a.num_pages == 0 || a.page_size == 0) return TOPK_OK;
  if (a.num_pages > INT64_MAX / a.page_size) return TOPK_EINVAL;
  if (a.k == nullptr || a.k_cache == nullptr || a.slots == nullptr || (values && a.v_cache == nullptr)) return TOPK_EINVAL;
  if (a.rotated > 0 && (a.positions == nullptr || a.frequencies == nullptr)) return TOPK_EINVAL;
  if (scaled && (a.k_scales == nullptr || (values && a.v_scales == nullptr))) return TOPK_EINVAL;
  unused(a.T, a.k_token_stride, a.v_token_stride);
  unused(a.H, a.k_head_stride, a.v_head_stride, a.k_cache_head_stride, a.v_cache_head_stride);
  unused(a.num_pages, a.k_cache_page_stride, a.v_cache_page_stride);
  unused(a.page_size, a.k_cache_token_stride, a.v_cache_token_stride);
  const uintptr_t size = static_cast<uintptr_t>(size_of(a.type)), cached = static_cast<uintptr_t>(size_of(a.cache_type));
  if (!aligned(a.k, size) || !aligned(a.k_cache, cached) || !aligned(a.slots, 4)) return TOPK_EINVAL;
  if (values && (!aligned(a.v, size) || !aligned(a.v_cache, cached))) return TOPK_EINVAL;
  if (a.rotated > 0 && (!aligned(a.positions, a.positions_64 ? 8 : 4) || !aligned(a.frequencies, 8))) return TOPK_EINVAL;
  if (scaled && (!aligned(a.k_scales, 4) || (values && !aligned(a.v_scales, 4)))) return TOPK_EINVAL;
  int dev = 0, sms = 0;
  const topk_status st = ready(&dev, &sms);
  if (st != TOPK_OK) return st;
  return launch_append(a, sms, reinterpret_cast<cudaStream_t>(stream));
}

topk_status sparse_attention_e4m3(const sparse_attention_e4m3_args* args, topk_stream_t stream) {
  if (args == nullptr) return TOPK_EINVAL;
  sparse_attention_e4m3_args all = *args;
  sparse_attention_args& a = all.attention;
  if (a.type != SPARSE_BF16 && a.type != SPARSE_FP16) return TOPK_EINVAL;
  if (a.B < 0 || a.T < 0 || a.Hkv < 1 || a.Hq < 0 || a.Hq % a.Hkv != 0 || a.K < 0) return TOPK_EINVAL;
  if (a.D < 16 || a.D > SPARSE_ATTENTION_MAX_D || a.D % 16 != 0) return TOPK_EINVAL;
  if (a.Dv < 16 || a.Dv > SPARSE_ATTENTION_MAX_D || a.Dv % 16 != 0) return TOPK_EINVAL;
  if (!std::isfinite(a.scale) || !std::isfinite(a.softcap) || a.softcap < 0.0f) return TOPK_EINVAL;
  if (a.num_pages < 0 || a.page_size < 0 || a.table_width < 0 || a.table_stride < 0) return TOPK_EINVAL;
  if (a.page_size > 0 && (all.blocks < 1 || a.page_size % all.blocks != 0)) return TOPK_EINVAL;
  if (a.page_table == nullptr && (a.query_positions != nullptr || a.first != nullptr || a.slopes != nullptr))
    return TOPK_EINVAL;
  if (a.slopes != nullptr && a.query_positions == nullptr) return TOPK_EINVAL;
  if (a.B == 0 || a.T == 0 || a.Hq == 0) return TOPK_OK;
  if (a.page_size > 0 && a.num_pages > INT64_MAX / a.page_size) return TOPK_EINVAL;
  const int64_t rows = static_cast<int64_t>(a.B) * a.T, heads = a.Hq / a.Hkv;
  if (rows > INT32_MAX || rows * a.Hkv > INT32_MAX || rows * a.Hkv * ((heads + 7) / 8) > INT32_MAX) return TOPK_EINVAL;
  const bool entries = a.K > 0 && a.num_pages > 0 && a.page_size > 0;
  if (a.q == nullptr || a.out == nullptr || (a.K > 0 && a.indices == nullptr)) return TOPK_EINVAL;
  if (entries && (a.k == nullptr || a.v == nullptr || all.k_scales == nullptr || all.v_scales == nullptr)) return TOPK_EINVAL;
  unused(a.B, a.q_seq_stride, a.table_stride);
  unused(a.T, a.q_token_stride);
  unused(a.Hq, a.q_head_stride);
  unused(a.num_pages, a.k_page_stride, a.v_page_stride);
  unused(a.page_size, a.k_token_stride, a.v_token_stride);
  unused(a.Hkv, a.k_head_stride, a.v_head_stride);
  if (!aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.out, 16) || !aligned(a.q, 2)) return TOPK_EINVAL;
  for (const int64_t s : {a.k_page_stride, a.k_token_stride, a.k_head_stride, a.v_page_stride, a.v_token_stride,
                          a.v_head_stride})
    if (!whole16(s, 1)) return TOPK_EINVAL;
  if (!aligned(a.indices, 4) || !aligned(a.page_table, 4) || !aligned(a.query_positions, 4) || !aligned(a.first, 4) ||
      !aligned(a.slopes, 4) || !aligned(a.lse, 4) || !aligned(all.k_scales, 4) || !aligned(all.v_scales, 4))
    return TOPK_EINVAL;
  int dev = 0, sms = 0;
  const topk_status st = ready(&dev, &sms);
  if (st != TOPK_OK) return st;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return a.type == SPARSE_BF16 ? launch_cache_attention_bf16(all, dev, sms, cs) : launch_cache_attention_fp16(all, dev, sms, cs);
}

}  // extern "C"
