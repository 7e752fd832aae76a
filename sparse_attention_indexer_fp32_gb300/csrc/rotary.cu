// Rotary positions (include/sparse_step.h, sparse_rotary).
//
// The angle. With f_i radians per position, one position turns pair i by
// f_i / 2 pi turns; only the fraction of a turn counts. So the rate is held as
// a fixed-point fraction of a turn in 64 bits and multiplied by the position
// in integer arithmetic modulo 2^64: whole turns drop out by themselves and
// the fraction is exact up to the rate's rounding (2^-64 turns) times the
// position, 2^-33 turns at position 2^31, where a product in FP32 would be
// off by whole turns. Its top 32 bits go to sinpi / cospi as FP32.
//
// The work. Memory bound: each element is read and written once, with three
// operations. A CTA takes a few tokens and heads, 16 bytes per item; it first
// issues the loads of its first items, then fills a table of (cos, sin) of its
// tokens in shared memory, once for all of their heads, then turns and stores.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "step_launch.cuh"

namespace tki {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotUnroll = 4;        // items of one thread whose loads are in flight together
constexpr int kRotTable = 2048;      // (cos, sin) pairs of a CTA's tokens: 16 KiB
constexpr int kRotMaxPairs = SPARSE_ROTARY_MAX_D / 2;

struct RotParams {
  const void* x;
  int64_t x_token, x_head;
  void* out;
  int64_t out_page, out_token, out_head;
  const void* positions;
  const double* frequencies;
  const int32_t* slots;
  int64_t num_slots;
  int32_t page_size;
  int32_t T, H, D, rotated, offset;
  int32_t positions_64;
  int32_t turn_items, items;       // per head: items that turn pairs, and with those that copy
  int32_t tokens, heads;           // per CTA
  int32_t head_chunks;
  uint32_t inv_items, inv_heads;   // reciprocals for quotients of small numbers
  float scale, sign;
};

// e / d for e, d < 2^16 and inv = floor(2^32 / d) + 1 (0 stands for d = 1).
__device__ __forceinline__ uint32_t quotient(uint32_t e, uint32_t inv) { return inv == 0 ? e : __umulhi(e, inv); }

// f / 2 pi as a fraction of a turn, times 2^64, modulo 2^64. The mantissa m of
// f = m 2^(e - 1075) is multiplied by round(2^66 / 2 pi) into 117 bits and
// shifted.
__device__ __forceinline__ uint64_t turns_of(double f) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
  const int e = static_cast<int>((bits >> 52) & 0x7ff);
  if (e == 0) return 0;  // zero, or under 2^-1022
  const uint64_t m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
  const uint64_t c = 0xa2f9836e4e44152aull;
  const uint64_t lo = m * c, hi = __umul64hi(m, c);
  const int shift = 1077 - e;
  uint64_t t;
  if (shift <= 0)
    t = 0;  // 2^54 radians a position and more: outside the contract
  else if (shift < 64)
    t = (lo >> shift) | (hi << (64 - shift));
  else if (shift < 128)
    t = hi >> (shift - 64);
  else
    t = 0;
  return (bits >> 63) ? 0ull - t : t;
}

template <typename E>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};

template <typename E, int V>
struct alignas(sizeof(E) * V) Vec {
  E e[V];
};

// V elements per item side. HALF: an item that turns holds V elements of the
// first half and V of the second; otherwise V consecutive ones (V / 2 pairs;
// V = 2 where nothing is aligned). Items after `turn_items` copy V elements
// of the head's rest (one, where V is the unaligned variant's).
template <typename E, int V, bool HALF>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotParams p) {
  constexpr bool kVector = sizeof(E) * V == 16;
  constexpr int kCopy = kVector ? V : 1;
  using VecT = Vec<E, V>;
  __shared__ uint64_t rate[kRotMaxPairs];
  __shared__ float2 table[kRotTable];
  const int pairs = p.rotated / 2;
  const int64_t chunk = blockIdx.x;
  const int t0 = static_cast<int>(chunk / p.head_chunks) * p.tokens;
  const int h0 = static_cast<int>(chunk % p.head_chunks) * p.heads;
  const int nt = min(p.tokens, p.T - t0), nh = min(p.heads, p.H - h0);
  const int total = nt * p.heads * p.items;

  const E* xb[kRotUnroll];
  E* ob[kRotUnroll];
  VecT a[kRotUnroll], b[kRotUnroll];
  int item[kRotUnroll], tok[kRotUnroll];

  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < kRotUnroll; ++u) {
      const uint32_t e = base + u * kRotThreads + threadIdx.x;
      item[u] = -1;
      if (e >= static_cast<uint32_t>(total)) continue;
      const uint32_t th = quotient(e, p.inv_items);
      const int i = static_cast<int>(e - th * p.items);
      const uint32_t tt = quotient(th, p.inv_heads);
      const int hh = static_cast<int>(th - tt * p.heads);
      if (hh >= nh) continue;
      const int64_t t = t0 + static_cast<int>(tt), h = h0 + hh;
      E* o;
      if (p.slots != nullptr) {
        const int32_t s = p.slots[t];
        if (s < 0 || s >= p.num_slots) continue;
        const int32_t page = s / p.page_size;
        o = static_cast<E*>(p.out) + page * p.out_page + (s - page * p.page_size) * p.out_token + h * p.out_head;
      } else {
        o = static_cast<E*>(p.out) + t * p.out_token + h * p.out_head;
      }
      const E* x = static_cast<const E*>(p.x) + t * p.x_token + h * p.x_head;
      item[u] = i;
      tok[u] = static_cast<int>(tt);
      int at;
      if (i < p.turn_items) {
        at = p.offset + i * (HALF && !kVector ? 1 : V);
        if constexpr (kVector) {
          a[u] = *reinterpret_cast<const VecT*>(x + at);
          if (HALF) b[u] = *reinterpret_cast<const VecT*>(x + at + pairs);
        } else {
          a[u].e[0] = x[at];
          a[u].e[1] = x[at + (HALF ? pairs : 1)];
        }
      } else {
        at = (i - p.turn_items) * kCopy;
        if (at >= p.offset) at += p.rotated;
        if constexpr (kVector)
          a[u] = *reinterpret_cast<const VecT*>(x + at);
        else
          a[u].e[0] = x[at];
      }
      xb[u] = x;
      ob[u] = o + at;
    }
  };

  auto store = [&]() {
#pragma unroll
    for (int u = 0; u < kRotUnroll; ++u) {
      if (item[u] < 0) continue;
      E* o = ob[u];
      if (item[u] >= p.turn_items) {
        if constexpr (kVector)
          *reinterpret_cast<VecT*>(o) = a[u];
        else
          o[0] = a[u].e[0];
        continue;
      }
      if constexpr (!kVector) {
        const float2 cs = table[tok[u] * pairs + item[u]];
        const float r = Elem<E>::get(a[u].e[0]), s = Elem<E>::get(a[u].e[1]);
        o[0] = Elem<E>::put(r * cs.x - s * cs.y);
        o[HALF ? pairs : 1] = Elem<E>::put(s * cs.x + r * cs.y);
      } else if constexpr (HALF) {
        const float2* cs = table + tok[u] * pairs + item[u] * V;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float2 c = cs[j];
          const float r = Elem<E>::get(a[u].e[j]), s = Elem<E>::get(b[u].e[j]);
          a[u].e[j] = Elem<E>::put(r * c.x - s * c.y);
          b[u].e[j] = Elem<E>::put(s * c.x + r * c.y);
        }
        *reinterpret_cast<VecT*>(o) = a[u];
        *reinterpret_cast<VecT*>(o + pairs) = b[u];
      } else {
        const float2* cs = table + tok[u] * pairs + item[u] * (V / 2);
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          const float2 c = cs[j / 2];
          const float r = Elem<E>::get(a[u].e[j]), s = Elem<E>::get(a[u].e[j + 1]);
          a[u].e[j] = Elem<E>::put(r * c.x - s * c.y);
          a[u].e[j + 1] = Elem<E>::put(s * c.x + r * c.y);
        }
        *reinterpret_cast<VecT*>(o) = a[u];
      }
    }
  };

  load(0);
  for (int i = threadIdx.x; i < pairs; i += kRotThreads) rate[i] = turns_of(p.frequencies[i]);
  __syncthreads();
  for (int e = threadIdx.x; e < nt * pairs; e += kRotThreads) {
    const int tt = e / pairs, i = e - tt * pairs;
    const int64_t pos = p.positions_64 ? static_cast<const int64_t*>(p.positions)[t0 + tt]
                                       : static_cast<const int32_t*>(p.positions)[t0 + tt];
    const uint64_t turn = static_cast<uint64_t>(pos) * rate[i];
    const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    table[e] = make_float2(c * p.scale, s * p.sign);
  }
  __syncthreads();
  store();
  for (int base = kRotUnroll * kRotThreads; base < total; base += kRotUnroll * kRotThreads) {
    load(base);
    store();
  }
}

template <typename E>
topk_status launch_typed(const sparse_rotary_args& a, int sm_count, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(E);
  const bool half = a.layout == SPARSE_ROTARY_HALF;
  auto whole = [](int64_t n) { return n % V == 0; };
  auto aligned16 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  // 16-byte items need every item to start on 16 bytes; otherwise one pair
  // (or one copied element) an item.
  const bool vec = aligned16(a.x) && aligned16(a.out) && whole(a.x_token_stride) && whole(a.x_head_stride) &&
                   whole(a.out_token_stride) && whole(a.out_head_stride) &&
                   (a.slots == nullptr || whole(a.out_page_stride)) && whole(a.D) && whole(a.offset) &&
                   whole(half ? a.rotated / 2 : a.rotated);
  // In place the rest of the head is already there.
  const bool in_place = a.slots == nullptr && a.x == a.out && a.x_token_stride == a.out_token_stride &&
                        a.x_head_stride == a.out_head_stride;
  RotParams p = {};
  p.x = a.x, p.x_token = a.x_token_stride, p.x_head = a.x_head_stride;
  p.out = a.out, p.out_page = a.out_page_stride, p.out_token = a.out_token_stride, p.out_head = a.out_head_stride;
  p.positions = a.positions, p.frequencies = a.frequencies, p.slots = a.slots;
  p.num_slots = a.slots != nullptr ? a.num_pages * a.page_size : 0;
  p.page_size = a.page_size;
  p.T = a.T, p.H = a.H, p.D = a.D, p.rotated = a.rotated, p.offset = a.offset;
  p.positions_64 = a.positions_64;
  p.scale = a.scale, p.sign = a.inverse ? -a.scale : a.scale;
  const int pairs = a.rotated / 2;
  p.turn_items = vec ? (half ? pairs / V : a.rotated / V) : pairs;
  p.items = p.turn_items + (in_place ? 0 : (a.D - a.rotated) / (vec ? V : 1));
  // Items per CTA: four per thread, so that a thread's loads overlap, once
  // that still gives every SM several CTAs; one per thread below.
  const int64_t all = static_cast<int64_t>(a.T) * a.H * p.items;
  const int want = all >= static_cast<int64_t>(sm_count) * 8 * kRotThreads * kRotUnroll ? kRotThreads * kRotUnroll
                                                                                        : kRotThreads;
  p.heads = want / p.items < 1 ? 1 : (want / p.items < a.H ? want / p.items : a.H);
  p.tokens = want / (p.items * p.heads);
  if (p.tokens > kRotTable / pairs) p.tokens = kRotTable / pairs;
  if (p.tokens > a.T) p.tokens = a.T;
  if (p.tokens < 1) p.tokens = 1;
  p.head_chunks = (a.H + p.heads - 1) / p.heads;
  auto reciprocal = [](int d) { return d == 1 ? 0u : static_cast<uint32_t>((1ull << 32) / static_cast<unsigned>(d)) + 1u; };
  p.inv_items = reciprocal(p.items);
  p.inv_heads = reciprocal(p.heads);
  const int64_t grid = static_cast<int64_t>((a.T + p.tokens - 1) / p.tokens) * p.head_chunks;
  if (grid > INT32_MAX) return TOPK_EINVAL;
  const unsigned g = static_cast<unsigned>(grid);
  if (vec)
    half ? rotary_kernel<E, V, true><<<g, kRotThreads, 0, stream>>>(p)
         : rotary_kernel<E, V, false><<<g, kRotThreads, 0, stream>>>(p);
  else
    half ? rotary_kernel<E, 2, true><<<g, kRotThreads, 0, stream>>>(p)
         : rotary_kernel<E, 2, false><<<g, kRotThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? TOPK_OK : TOPK_ECUDA;
}

}  // namespace

topk_status launch_rotary(const sparse_rotary_args& a, int sm_count, cudaStream_t stream) {
  switch (a.type) {
    case SPARSE_BF16: return launch_typed<__nv_bfloat16>(a, sm_count, stream);
    case SPARSE_FP16: return launch_typed<__half>(a, sm_count, stream);
    default: return launch_typed<float>(a, sm_count, stream);
  }
}

}  // namespace tki
