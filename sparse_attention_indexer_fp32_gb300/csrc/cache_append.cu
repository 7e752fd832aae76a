// Keys and values into a paged cache (include/sparse_cache.h, sparse_append).
//
// The scale. A block's scale bounds its entries through |u| + |v| of each pair
// that turns, which holds at any angle: no rotation is needed to find it, it does
// not depend on the position, and one rounded sum gives the same bits in any
// order. It is a power of two, so that units change exactly: a block whose scale
// grows is multiplied by a power of two and rounded again only below E4M3's
// smallest normal number.
//
// The work. Memory bound: each element is read once and written once, in half or
// a quarter of its size. The tokens of a block follow one another, so a CTA takes
// the runs of tokens that begin in its share of the call, whole, for up to four
// heads of one side (keys or values): it finds the runs from the slots alone, the
// largest size of each run and head by an integer maximum in shared memory
// (sizes are not negative), then reads its tokens again from L1, turns and rounds
// them. No atomics to memory, no workspace; every block's scale has one writer.
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "cache_launch.cuh"
#include "e4m3.cuh"
#include "rotary_math.cuh"
#include "step_launch.cuh"

namespace tki {
namespace {

constexpr int kThreads = 256;
constexpr int kRuns = 64;  // tokens whose runs a CTA takes, so runs of a CTA

struct AppendSide {
  const void* x;
  int64_t x_token, x_head;
  void* cache;
  int64_t page, entry, head;
  float* scales;
  int32_t D, rotated, offset;
  int32_t turn_items, items;  // of a head: items that turn pairs, and with those that do not
  bool vector;                // 16-byte items; otherwise a pair, or one element, each
  bool rows16;                // entries of the cache in whole 16-byte units
};

struct AppendParams {
  AppendSide side[2];
  const void* positions;
  const double* frequencies;
  const int32_t* slots;
  int64_t num_slots;
  int32_t page_size, block;
  int32_t T, H;
  int32_t positions_64;
  int32_t head_groups;
  int32_t share;  // tokens whose runs a CTA takes; without scales, its tokens
  float scale;
};

struct AppendShared {
  uint64_t rates[SPARSE_APPEND_MAX_D / 2];  // of the pairs, in turns a position
  unsigned long long leads;                 // bit per token of the share: it begins a run
  int64_t end;                              // of the last run
  int32_t first[kRuns], block[kRuns];       // of a run: least place, and block of the cache
  uint32_t size[kThreads];                  // of a run and head: the largest size / 2, as its bits
  float unit[kThreads], ratio[kThreads];    // 1 / scale; what its earlier entries are multiplied by
};

// The smallest power of two s >= 2^-126 with 2 half <= 448 s = 1.75 2^8 s.
__device__ __forceinline__ float scale_for(float half) {
  const uint32_t bits = __float_as_uint(half);
  const int e = static_cast<int>(bits >> 23) - 127;
  const int n = e - 7 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(n, -126) + 127) << 23);
}

// One side of a CTA. V elements an item side; items and layouts as in rotary.cu,
// V = 2 where nothing is aligned.
template <typename E, int V, bool HALF, bool SCALED, int U>
__device__ __forceinline__ void append_side(const AppendParams& p, const AppendSide& s, AppendShared& sh, bool turns_any) {
  constexpr bool kVector = sizeof(E) * V == 16;
  constexpr int kPairs = !kVector ? 1 : HALF ? V : V / 2;  // of an item
  using VecT = Vec<E, V>;
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t share = blockIdx.x / static_cast<unsigned>(p.head_groups);
  const int h0 = static_cast<int>(blockIdx.x - share * p.head_groups) * U;
  const int heads = min(p.H - h0, U);
  const int64_t t0 = share * p.share, t1 = min(t0 + p.share, static_cast<int64_t>(p.T));
  const int per = min(s.items, kThreads);
  const int sub = tid / per, i0 = tid - sub * per, side_by_side = kThreads / per;
  auto slot_of = [&](int64_t t) -> int32_t {  // -1: not written
    const int32_t slot = p.slots[t];
    return slot >= 0 && slot < p.num_slots ? slot : -1;
  };
  auto block_of = [&](int64_t t) -> int32_t {
    const int32_t slot = slot_of(t);
    return slot < 0 ? -1 : slot / p.block;
  };

  if (turns_any)
    for (int i = tid; i < s.rotated / 2; i += kThreads) sh.rates[i] = turns_of(p.frequencies[i]);
  int64_t begin = t0, end = t1;
  unsigned long long leads = 0;
  int runs = 0;
  float before = 0.0f;  // the scale that this thread's run and head has
  if constexpr (SCALED) {
    sh.size[tid] = 0;
    if (tid < kRuns) sh.first[tid] = INT32_MAX;
    if (tid < 32) {
#pragma unroll
      for (int part = 0; part < kRuns; part += 32) {
        const int64_t t = t0 + part + lane;
        const int32_t block = t < t1 ? block_of(t) : -1;
        const bool lead = block >= 0 && (t == 0 || block_of(t - 1) != block);
        const uint32_t bits = __ballot_sync(0xffffffffu, lead);
        if (lead) sh.block[__popcll(leads) + __popc(bits & ((1u << lane) - 1))] = block;
        leads |= static_cast<unsigned long long>(bits) << part;
      }
      if (leads != 0) {  // the last run may go on behind the share
        const int32_t last = block_of(t1 - 1);
        while (last >= 0) {
          const bool on = end + lane < p.T && block_of(end + lane) == last;
          const uint32_t off = ~__ballot_sync(0xffffffffu, on);
          end += off != 0 ? __ffs(off) - 1 : 32;
          if (off != 0) break;
        }
      }
      if (tid == 0) sh.leads = leads, sh.end = end;
    }
    __syncthreads();
    leads = sh.leads, end = sh.end;
    if (leads == 0) return;
    runs = __popcll(leads);
    begin = t0 + __ffsll(static_cast<long long>(leads)) - 1;
    const int r = tid / U;
    if (r < runs && tid % U < heads) before = s.scales[static_cast<int64_t>(sh.block[r]) * p.H + h0 + tid % U];
  } else {
    __syncthreads();
  }
  // The run of a token between begin and end that is written.
  auto run_of = [&](int64_t t) { return t < t1 ? __popcll(leads & ((2ull << (t - t0)) - 1)) - 1 : runs - 1; };

  // An item of a token's head.
  const E* x = static_cast<const E*>(s.x) + h0 * s.x_head;
  const int pairs = s.rotated / 2;
  const int partner = HALF ? pairs : 1;  // of the unaligned item's first element
  auto place_of = [&](int i) {
    if (i < s.turn_items) return s.offset + i * (HALF && !kVector ? 1 : V);
    const int at = (i - s.turn_items) * (kVector ? V : 1);
    return at >= s.offset && s.rotated > 0 ? at + s.rotated : at;
  };
  auto load = [&](const E* from, bool turns, VecT& a, VecT& b) {
    if constexpr (kVector) {
      a = load16<VecT>(from);
      if (HALF && turns) b = load16<VecT>(from + pairs);
    } else {
      a.e[0] = from[0];
      if (turns) a.e[1] = from[partner];
    }
  };

  if constexpr (SCALED) {
    // ---- the largest sizes ----
    for (int64_t t = begin + sub; sub < side_by_side && t < end; t += side_by_side) {
      const int32_t slot = slot_of(t);
      if (slot < 0) continue;
      const int run = run_of(t);
      if (i0 == 0) atomicMin(&sh.first[run], slot % p.block);
      for (int i = i0; i < s.items; i += per) {
        const bool turns = i < s.turn_items;
        const E* from = x + t * s.x_token + place_of(i);
        VecT a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < heads) load(from + u * s.x_head, turns, a[u], b[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u >= heads) continue;
          float most = 0.0f;
          auto count = [&](float size) {  // a NaN or an infinity does not count
            if (size <= FLT_MAX) most = fmaxf(most, size);
          };
          auto half = [](E e) { return 0.5f * fabsf(Elem<E>::get(e)); };
          if (turns) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
              const E second = HALF && kVector ? b[u].e[j] : a[u].e[2 * j + 1];
              count((half(a[u].e[HALF ? j : 2 * j]) + half(second)) * fabsf(p.scale));
            }
          } else {
#pragma unroll
            for (int j = 0; j < (kVector ? V : 1); ++j) count(half(a[u].e[j]));
          }
          atomicMax(&sh.size[run * U + u], __float_as_uint(most));
        }
      }
    }
    __syncthreads();
    // ---- the scales ----
    const int r = tid / U;
    if (r < runs && tid % U < heads) {
      const float need = scale_for(__uint_as_float(sh.size[tid]));
      const bool begins = sh.first[r] == 0;
      const float now = begins ? need : fmaxf(before, need);
      if (begins || now != before) s.scales[static_cast<int64_t>(sh.block[r]) * p.H + h0 + tid % U] = now;
      sh.unit[tid] = 1.0f / now;
      sh.ratio[tid] = begins ? 1.0f : before / now;
    }
    __syncthreads();
  }

  // ---- the tokens ----
  for (int64_t t = begin + sub; sub < side_by_side && t < end; t += side_by_side) {
    const int32_t slot = slot_of(t);
    if (slot < 0) continue;
    const int32_t page = slot / p.page_size;
    const int64_t entry = page * s.page + (slot - page * p.page_size) * s.entry + h0 * s.head;
    const int run = SCALED ? run_of(t) : 0;
    for (int i = i0; i < s.items; i += per) {
      const bool turns = i < s.turn_items;
      const int at = place_of(i);
      const E* from = x + t * s.x_token + at;
      VecT a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < heads) load(from + u * s.x_head, turns, a[u], b[u]);
      float cosines[kPairs], sines[kPairs];
      if (turns) {
        const int64_t pos = p.positions_64 ? static_cast<const int64_t*>(p.positions)[t] : static_cast<const int32_t*>(p.positions)[t];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const uint64_t turn = static_cast<uint64_t>(pos) * sh.rates[i * kPairs + j];
          const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
          // 2^-21 by the special function unit: 2^-10 of a 16-bit result's
          // rounding, 2^-17 of an 8-bit one's; FP32 takes the full functions.
          if constexpr (SCALED || sizeof(E) == 2)
            __sincosf(half_turns * 3.14159265f, &sines[j], &cosines[j]);
          else
            sincospif(half_turns, &sines[j], &cosines[j]);
          cosines[j] *= p.scale, sines[j] *= p.scale;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u >= heads) continue;
        float y[V], z[V];  // the item's elements, and with HALF their partners
        if constexpr (kVector) {
#pragma unroll
          for (int j = 0; j < V; ++j) y[j] = Elem<E>::get(a[u].e[j]), z[j] = HALF ? Elem<E>::get(b[u].e[j]) : 0.0f;
        } else {
          y[0] = Elem<E>::get(a[u].e[0]), y[1] = turns ? Elem<E>::get(a[u].e[1]) : 0.0f;
        }
        if (turns) {
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            float& first = y[HALF ? j : 2 * j];
            float& second = HALF && kVector ? z[j] : y[2 * j + 1];
            const float r = first, q = second;
            first = r * cosines[j] - q * sines[j];
            second = q * cosines[j] + r * sines[j];
          }
        }
        if constexpr (SCALED) {
          uint8_t* to = static_cast<uint8_t*>(s.cache) + entry + u * s.head + at;
          const float unit = sh.unit[run * U + u];
          // a product with 0 is 0, or NaN of what is not finite
          auto two = [&](float m, float n) { return e4m3_two(fmaf(m, unit, m * 0.0f), fmaf(n, unit, n * 0.0f)); };
          if constexpr (kVector) {
            auto put = [&](uint8_t* to, const float(&y)[V]) {
              uint32_t w[V / 4];
#pragma unroll
              for (int j = 0; j < V; j += 4) w[j / 4] = two(y[j], y[j + 1]) | two(y[j + 2], y[j + 3]) << 16;
              if constexpr (V == 8)
                *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
              else
                *reinterpret_cast<uint32_t*>(to) = w[0];
            };
            put(to, y);
            if (HALF && turns) put(to + pairs, z);
          } else {
            const uint32_t w = two(y[0], y[1]);
            to[0] = static_cast<uint8_t>(w);
            if (turns) to[partner] = static_cast<uint8_t>(w >> 8);
          }
        } else {
          E* to = static_cast<E*>(s.cache) + entry + u * s.head + at;
          if constexpr (kVector) {
            VecT c;
#pragma unroll
            for (int j = 0; j < V; ++j) c.e[j] = Elem<E>::put(y[j]);
            store16(to, c);
            if (HALF && turns) {
#pragma unroll
              for (int j = 0; j < V; ++j) c.e[j] = Elem<E>::put(z[j]);
              store16(to + pairs, c);
            }
          } else {
            to[0] = Elem<E>::put(y[0]);
            if (turns) to[partner] = Elem<E>::put(y[1]);
          }
        }
      }
    }
  }

  if constexpr (SCALED) {
    // ---- earlier entries of blocks whose scale grew, one run and head a warp ----
    for (int j = tid >> 5; j < runs * U; j += kThreads / 32) {
      const int r = j / U, u = j - r * U;
      if (u >= heads || sh.ratio[j] == 1.0f) continue;
      const float ratio = sh.ratio[j];
      const int32_t block = sh.block[r], per_page = p.page_size / p.block, page = block / per_page;
      uint8_t* base = static_cast<uint8_t*>(s.cache) + page * s.page +
                      static_cast<int64_t>(block - page * per_page) * p.block * s.entry + (h0 + u) * s.head;
      const int rows = sh.first[r];
      auto again = [&](uint32_t two) {
        const float2 v = e4m3_both(two);
        return e4m3_two(v.x * ratio, v.y * ratio);
      };
      if (s.rows16) {
        const int row_units = s.D / 16;
        const int64_t units = static_cast<int64_t>(rows) * row_units;
        constexpr int kAhead = 8;
        for (int64_t n = lane; n < units; n += 32 * kAhead) {
          uint4 v[kAhead];
          uint4* from[kAhead];
#pragma unroll
          for (int a = 0; a < kAhead; ++a) {
            const int64_t at = n + a * 32, row = at / row_units;
            from[a] = reinterpret_cast<uint4*>(base + row * s.entry) + (at - row * row_units);
            if (at < units) v[a] = *from[a];
          }
#pragma unroll
          for (int a = 0; a < kAhead; ++a) {
            if (n + a * 32 >= units) continue;
            uint32_t* w = reinterpret_cast<uint32_t*>(&v[a]);
#pragma unroll
            for (int c = 0; c < 4; ++c) w[c] = again(w[c] & 0xffff) | again(w[c] >> 16) << 16;
            *from[a] = v[a];
          }
        }
      } else {
        for (int64_t n = lane; n < static_cast<int64_t>(rows) * s.D; n += 32) {
          const int64_t row = n / s.D;
          uint8_t* at = base + row * s.entry + (n - row * s.D);
          *at = static_cast<uint8_t>(again(*at));
        }
      }
    }
  }
}

template <typename E, bool HALF, bool SCALED, int U>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ AppendShared sh;
  const AppendSide& s = p.side[blockIdx.y];
  if (s.vector)
    append_side<E, 16 / sizeof(E), HALF, SCALED, U>(p, s, sh, s.rotated > 0);
  else
    append_side<E, 2, HALF, SCALED, U>(p, s, sh, s.rotated > 0);
}

bool aligned_to(const void* q, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(q) & (bytes - 1)) == 0; }

template <typename E, bool HALF, bool SCALED>
topk_status launch_layout(const AppendParams& p, int sides, int sm_count, cudaStream_t stream) {
  AppendParams q = p;
  auto groups = [&](int share, int u) { return ((static_cast<int64_t>(p.T) + share - 1) / share) * ((p.H + u - 1) / u); };
  // Four heads a thread share their tokens' angles and have their loads in
  // flight together; one where that leaves SMs idle.
  int most = 1;  // tokens of one CTA side by side
  for (int i = 0; i < sides; ++i) {
    const int per = q.side[i].items < kThreads ? q.side[i].items : kThreads;
    if (kThreads / per > most) most = kThreads / per;
  }
  int share = kRuns;
  const bool four = groups(share, 4) * sides >= 2 * sm_count;
  const int u = four ? 4 : 1;
  while (share > 1 && groups(share, u) * sides < sm_count) share /= 2;
  if (!SCALED)
    while (share > 1 && share > most) share /= 2;
  q.share = share;
  q.head_groups = (p.H + u - 1) / u;
  const int64_t grid = groups(share, u);
  if (grid > INT32_MAX) return TOPK_EINVAL;
  const dim3 g(static_cast<unsigned>(grid), static_cast<unsigned>(sides));
  return launch(four ? append_kernel<E, HALF, SCALED, 4> : append_kernel<E, HALF, SCALED, 1>, q, g, kThreads, 0, stream);
}

template <typename E>
topk_status launch_typed(const sparse_append_args& a, int sm_count, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(E);
  const bool scaled = a.cache_type == SPARSE_E4M3, half = a.layout == SPARSE_ROTARY_HALF;
  const int64_t size = scaled ? 1 : static_cast<int64_t>(sizeof(E));  // of a cache's element
  auto whole = [](int64_t n) { return n % V == 0; };
  AppendParams p = {};
  p.positions = a.positions, p.frequencies = a.frequencies, p.slots = a.slots;
  p.num_slots = a.num_pages * a.page_size;
  p.page_size = a.page_size, p.block = scaled ? a.page_size / a.blocks : 1;
  p.T = a.T, p.H = a.H, p.positions_64 = a.positions_64, p.scale = a.scale;
  const int sides = a.v != nullptr ? 2 : 1;
  for (int i = 0; i < sides; ++i) {
    AppendSide& s = p.side[i];
    const bool keys = i == 0;
    s.x = keys ? a.k : a.v, s.x_token = keys ? a.k_token_stride : a.v_token_stride, s.x_head = keys ? a.k_head_stride : a.v_head_stride;
    s.cache = keys ? a.k_cache : a.v_cache, s.scales = keys ? a.k_scales : a.v_scales;
    s.page = keys ? a.k_cache_page_stride : a.v_cache_page_stride;
    s.entry = keys ? a.k_cache_token_stride : a.v_cache_token_stride;
    s.head = keys ? a.k_cache_head_stride : a.v_cache_head_stride;
    s.D = keys ? a.D : a.Dv, s.rotated = keys ? a.rotated : 0, s.offset = keys ? a.offset : 0;
    s.vector = aligned_to(s.x, 16) && aligned_to(s.cache, static_cast<uintptr_t>(V * size)) && whole(s.x_token) && whole(s.x_head) &&
               whole(s.page) && whole(s.entry) && whole(s.head) && whole(s.D) && whole(s.offset) &&
               whole(half ? s.rotated / 2 : s.rotated);
    const int pairs = s.rotated / 2;
    s.turn_items = s.vector ? (half ? pairs / V : s.rotated / V) : pairs;
    s.items = s.turn_items + (s.D - s.rotated) / (s.vector ? V : 1);
    s.rows16 = aligned_to(s.cache, 16) && s.page % 16 == 0 && s.entry % 16 == 0 && s.head % 16 == 0 && s.D % 16 == 0;
  }
  if (scaled) return half ? launch_layout<E, true, true>(p, sides, sm_count, stream) : launch_layout<E, false, true>(p, sides, sm_count, stream);
  return half ? launch_layout<E, true, false>(p, sides, sm_count, stream) : launch_layout<E, false, false>(p, sides, sm_count, stream);
}

}  // namespace

topk_status launch_append(const sparse_append_args& a, int sm_count, cudaStream_t stream) {
  switch (a.type) {
    case SPARSE_BF16: return launch_typed<__nv_bfloat16>(a, sm_count, stream);
    case SPARSE_FP16: return launch_typed<__half>(a, sm_count, stream);
    default: return launch_typed<float>(a, sm_count, stream);
  }
}

}  // namespace tki
