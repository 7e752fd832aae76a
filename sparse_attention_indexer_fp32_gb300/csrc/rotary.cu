// Rotary positions (include/sparse_step.h, sparse_rotary).
//
// The angle. With f_i radians per position, one position turns pair i by
// f_i / 2 pi turns; only the fraction of a turn counts. So the rate is held as
// a fixed-point fraction of a turn in 64 bits and multiplied by the position
// in integer arithmetic modulo 2^64: whole turns drop out by themselves and
// the fraction is exact up to the rate's rounding (2^-63 turns) times the
// position, 2^-32 turns at position 2^31, where a product in FP32 would be
// off by whole turns. Its top 32 bits go to the trigonometric functions as FP32.
//
// The work. Memory bound: each element is read and written once, with three
// operations. A thread owns one 16-byte item of the head (two, where the
// second half's partner goes with it) of one token and walks over heads, so
// that it computes its pairs' cos and sin once, in registers, while its first
// loads are in flight; no shared memory, no barrier (a table per CTA in shared
// memory puts two barriers between loads and stores, and took twice as long).
//
// Measured: 8192 tokens x 64 heads x 128, bf16, 41.7 us, 6.4 TB/s, against 39.5 us
// for its bytes at the measured copy rate; 4097 x 24 x 80 in FP32 8.0 us, partly
// from L2 (9.3 from HBM); four tokens 3.5 us, most of it the launch and three
// dependent reads. 2048 x 64 x 130, where nothing is aligned, 23.5 us for 9.6 of
// the 128: two bytes an access.
#include <cuda_runtime.h>

#include <cstdint>

#include "rotary_math.cuh"
#include "step_launch.cuh"

namespace tki {
namespace {

constexpr int kRotThreads = 256;

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
  int32_t turn_items, items;  // per head: items that turn pairs, and with those that copy
  int32_t rows;               // rows (a token's head) that a CTA has side by side
  int32_t tokens, heads;      // tokens per CTA, heads of each side by side: tokens * heads <= rows
  int32_t head_span;          // heads per CTA, in steps of `heads`
  int32_t head_chunks;
  float scale, sign;
};

// V elements per item side. HALF: an item that turns holds V elements of the
// first half and V of the second; otherwise V consecutive ones (V / 2 pairs).
// V = 2 where nothing is aligned: one pair, or one copied element, an item.
template <typename E, int V, bool HALF>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotParams p) {
  constexpr bool kVector = sizeof(E) * V == 16;
  constexpr int kRotUnroll = HALF ? 2 : 4;  // heads whose loads are in flight together: 64 bytes
  constexpr int kPairs = !kVector ? 1 : HALF ? V : V / 2;  // of an item
  using VecT = Vec<E, V>;
  const int n = min(p.items, kRotThreads);
  const int sub = threadIdx.x / n;
  const int i = blockIdx.y * kRotThreads + (threadIdx.x - sub * n);
  const int tsub = sub / p.heads;
  const unsigned group = blockIdx.x / static_cast<unsigned>(p.head_chunks);
  const int h0 = static_cast<int>(blockIdx.x - group * p.head_chunks) * p.head_span;
  const int64_t t = static_cast<int64_t>(group) * p.tokens + tsub;
  if (i >= p.items || tsub >= p.tokens || t >= p.T) return;
  const int pairs = p.rotated / 2;
  const bool turns = i < p.turn_items;
  int at;  // of the item in its head
  if (turns) {
    at = p.offset + i * (HALF && !kVector ? 1 : V);
  } else {
    at = (i - p.turn_items) * (kVector ? V : 1);
    if (at >= p.offset) at += p.rotated;
  }
  const E* x = static_cast<const E*>(p.x) + t * p.x_token + at;
  E* o;
  if (p.slots != nullptr) {
    const int32_t s = p.slots[t];
    if (s < 0 || s >= p.num_slots) return;
    const int32_t page = s / p.page_size;
    o = static_cast<E*>(p.out) + page * p.out_page + (s - page * p.page_size) * p.out_token + at;
  } else {
    o = static_cast<E*>(p.out) + t * p.out_token + at;
  }
  const int partner = HALF ? pairs : 1;  // of the unaligned item's first element

  VecT a[kRotUnroll], b[kRotUnroll];
  const int end = min(h0 + p.head_span, p.H);
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kRotUnroll; ++u) {
      const int hu = h + u * p.heads;
      if (hu >= end) break;
      const E* from = x + hu * p.x_head;
      if constexpr (kVector) {
        a[u] = load16<VecT>(from);
        if (HALF && turns) b[u] = load16<VecT>(from + pairs);
      } else {
        a[u].e[0] = from[0];
        if (turns) a[u].e[1] = from[partner];
      }
    }
  };
  int h = h0 + sub - tsub * p.heads;
  load(h);
  float cosines[kPairs], sines[kPairs];
  if (turns) {
    const int64_t pos = p.positions_64 ? static_cast<const int64_t*>(p.positions)[t] : static_cast<const int32_t*>(p.positions)[t];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const uint64_t turn = static_cast<uint64_t>(pos) * turns_of(p.frequencies[i * kPairs + j]);
      // Within half a turn either way the special function unit is good to
      // 2^-20 (the special function unit's 2^-21.2, and 2^-21.6 of the angle: its rounding, that of pi and of
      // their product), 2^-9 of fp16's rounding; FP32 takes the full functions.
      const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
      if constexpr (sizeof(E) == 2)
        __sincosf(half_turns * 3.14159265f, &sines[j], &cosines[j]);
      else
        sincospif(half_turns, &sines[j], &cosines[j]);
      cosines[j] *= p.scale, sines[j] *= p.sign;
    }
  }
  while (h < end) {
#pragma unroll
    for (int u = 0; u < kRotUnroll; ++u) {
      const int hu = h + u * p.heads;
      if (hu >= end) break;
      E* to = o + hu * p.out_head;
      if (turns) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          E& first = a[u].e[HALF ? j : 2 * j];
          E& second = HALF && kVector ? b[u].e[j] : a[u].e[2 * j + 1];
          const float r = Elem<E>::get(first), s = Elem<E>::get(second);
          first = Elem<E>::put(r * cosines[j] - s * sines[j]);
          second = Elem<E>::put(s * cosines[j] + r * sines[j]);
        }
      }
      if constexpr (kVector) {
        store16(to, a[u]);
        if (HALF && turns) store16(to + pairs, b[u]);
      } else {
        to[0] = a[u].e[0];
        if (turns) to[partner] = a[u].e[1];
      }
    }
    h += kRotUnroll * p.heads;
    if (h < end) load(h);
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
  // Heads per thread: as many as leave every SM a few CTAs, up to sixteen, so
  // that cos and sin are computed once for them (8192 tokens x 64 heads: 122 us by
  // one head, 72, 48, 42 and 42 by 2, 4, 8 and 16; four tokens: 3.5 us by one, 6.6 by 16).
  p.rows = p.items < kRotThreads ? kRotThreads / p.items : 1;
  const double threads = static_cast<double>(a.T) * a.H * p.items;
  const double slots = static_cast<double>(sm_count) * kRotThreads;
  const int steps = threads >= 64 * slots ? 16 : threads >= 32 * slots ? 8 : threads >= 16 * slots ? 4 : threads >= 8 * slots ? 2 : 1;
  p.heads = (a.H + steps - 1) / steps < p.rows ? (a.H + steps - 1) / steps : p.rows;
  p.tokens = p.rows / p.heads < a.T ? p.rows / p.heads : a.T;
  p.head_span = p.heads * steps;
  p.head_chunks = (a.H + p.head_span - 1) / p.head_span;
  const int64_t grid = (static_cast<int64_t>(a.T) + p.tokens - 1) / p.tokens * p.head_chunks;
  if (grid > INT32_MAX) return TOPK_EINVAL;
  const dim3 g(static_cast<unsigned>(grid), static_cast<unsigned>((p.items + kRotThreads - 1) / kRotThreads));
  const auto kernel = vec ? (half ? rotary_kernel<E, V, true> : rotary_kernel<E, V, false>)
                          : (half ? rotary_kernel<E, 2, true> : rotary_kernel<E, 2, false>);
  return launch(kernel, p, g, kRotThreads, 0, stream);
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
