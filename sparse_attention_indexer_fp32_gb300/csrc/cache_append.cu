// Keys and values into a paged cache (include/sparse_cache.h, sparse_append).
//
// The scale. A block's scale bounds its entries through |u| + |v| of each pair
// that turns, which holds at any angle: no rotation is needed to find it, it does
// not depend on the position, and one rounded sum gives the same bits in any
// order. It is a power of two, so that units change exactly: a block whose scale
// grows is multiplied by a power of two and rounded again only below E4M3's
// smallest normal number.
//
// The work. Each element is read once and written once, in half or a quarter of its
// size; the arithmetic on it takes longer than that, so what tokens and heads share is
// done once. The tokens of a block mostly follow one another, so a CTA takes the runs of
// tokens that begin in its share of the call, whole, for two heads of one side (keys or
// values): it finds the runs from the slots alone, the largest size of each run and head
// by an integer maximum in shared memory (sizes are not negative), then turns and
// rounds its tokens. A thread has 32 bytes of two tokens and two heads at once, in
// registers from the one step to the other where the CTA's tokens fit (a block of 64
// with heads of 128 does), read again from L1 otherwise; a token's sine and cosine serve
// both heads. No atomics to memory, no workspace; every block's scale has one writer.
//
// Any order. A block may have several runs, only where none fills it: a CTA with a run that does not
// looks through the call's other slots (a bit per hash of its blocks, eight slots a thread at once)
// and adds up the sizes of the tokens it finds, so that each run's CTA comes to the same scale; that
// of the first one writes it and what the block held before. This costs an ordered call 1.3 us with 64
// tokens, 4 with 8192 of four prompts (33.7; 29.8 without, wrong in other orders), 9 with 8192
// single tokens (43), where every CTA looks. Four tokens of each of 64 sequences step by step 16.4 us
// (9.6 in order); shuffled prompts cost their tokens squared (4 x 512 279 us, 4 x 2048 1090).
//
// Measured, in a CUDA graph: 8192 tokens x 8 heads x (128 + 128), bf16, into 8 bits 34 us for
// 7.4 at the copy rate. It is bound by instructions and by what they wait for: 26 an element,
// issue slots 41 % busy, DRAM 12 %; a CTA's three barriers (slots, sizes, scales) leave its
// warps idle where the CTA beside it has nothing to issue, and so do instructions that are not
// in the cache (2.2 of an issue's 13 cycles, 0.5 without the look through other slots). 4096 tokens x 8 x (128 + 128), fp16,
// as they are 10.4 us (4.8); 64 tokens 8.4 us, a launch and reads of slot, scale and token one
// behind the other; 8192 index keys of 128 with a scale each 8.3 us.
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "attention_math.cuh"
#include "cache_launch.cuh"
#include "e4m3.cuh"
#include "rotary_math.cuh"
#include "step_launch.cuh"

namespace tki {
namespace {

constexpr int kRuns = 64;      // tokens whose runs a CTA takes at most, so runs of a CTA
constexpr int kMostHeads = 4;  // of a CTA
constexpr int kMarks = 32768;  // for the blocks of a CTA's runs

struct AppendSide {
  const void* x;
  int64_t x_token, x_head;
  void* cache;
  int64_t page, entry, head;
  float* scales;
  int32_t D, rotated, offset;
  int32_t turn_items, items;  // of a head: items that turn pairs, and with those that do not
  bool vector;                // items of two 16-byte units; otherwise of a pair, or one element
  bool rows16;                // entries of the cache in whole 16-byte units
};

struct AppendParams {
  AppendSide side[2];
  const void* positions;
  const double* frequencies;
  const int32_t* slots;
  int64_t num_slots;
  int32_t page_size, block;
  int32_t page_shift, block_shift;  // log2, or -1
  int32_t T, H, head_groups;
  int32_t positions_64;
  int32_t share;  // tokens whose runs a CTA takes; without scales, its tokens
  float scale;
};

struct AppendShared {
  uint64_t rates[SPARSE_APPEND_MAX_D / 2];  // of the pairs, in turns a position
  int32_t first[kRuns], block[kRuns];       // of a run: the least place in its block, and that of the cache
  uint32_t size[kRuns * kMostHeads];        // of a run and head: the largest size / 2, as its bits; then 1 / scale
  float ratio[kRuns * kMostHeads];          // what its earlier entries are multiplied by
  uint4 marks[kMarks / 128];                // bit per hash of a block: a run may have it
  uint8_t same[kRuns], later[kRuns];        // the share's first run of the same block; whether a token of an earlier share has it
  bool parts, twice;                        // a run has not all of its block: others may have tokens of it; runs of this share may
  unsigned long long leads;                 // bit per token of the share: it begins a run
  int64_t end;                              // of the last run
};

// The smallest power of two s >= 2^-126 with 2 half <= 448 s = 1.75 2^8 s.
__device__ __forceinline__ float scale_for(float half) {
  const uint32_t bits = __float_as_uint(half);
  const int e = static_cast<int>(bits >> 23) - 127;
  const int n = e - 7 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(n, -126) + 127) << 23);
}

// The two numbers of 32 bits of a 16-bit type.
template <typename E>
__device__ __forceinline__ float2 floats_of(uint32_t two) {
  if constexpr (std::is_same<E, __half>::value)
    return __half22float2(*reinterpret_cast<const __half2*>(&two));
  else
    return make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
}

// What a CTA and its threads take.
template <int THREADS, int ROWS, int HEADS, int PER_SM, int SHARE>
struct FormOf {
  static constexpr int threads = THREADS, rows = ROWS, heads = HEADS, per_sm = PER_SM, share = SHARE;
};

// A thread's and a CTA's indices, read anew where they are wanted, so that nothing the compiler makes
// of them in find_runs takes registers from what follows.
__device__ __forceinline__ int thread_index() {
  int v;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(v));
  return v;
}
__device__ __forceinline__ uint32_t block_index() {
  uint32_t v;
  asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(v));
  return v;
}

// What a CTA takes: the first of its heads, their number, and the tokens whose runs it has.
struct Share {
  int h0, heads;
  int64_t t0, t1;
};
template <typename Form>
__device__ __forceinline__ Share share_of(const AppendParams& p) {
  const uint32_t at = block_index(), share = at / static_cast<uint32_t>(p.head_groups);
  Share c;
  c.h0 = static_cast<int>(at - share * p.head_groups) * Form::heads, c.heads = min(p.H - c.h0, Form::heads);
  c.t0 = static_cast<int64_t>(share) * p.share, c.t1 = min(c.t0 + p.share, static_cast<int64_t>(p.T));
  return c;
}

__device__ __forceinline__ int32_t slot_of(const AppendParams& p, int64_t t) {  // -1: not written
  const int32_t slot = p.slots[t];
  return slot >= 0 && slot < p.num_slots ? slot : -1;
}
__device__ __forceinline__ int32_t block_of(const AppendParams& p, int32_t slot) {
  return slot < 0 ? -1 : p.block_shift >= 0 ? slot >> p.block_shift : slot / p.block;
}

// The CTA's runs, into `sh`. Where a run does not fill its block, other runs may have tokens of that:
// each share that has some finds the same scale, from all of them, and the first one writes it and what
// the block held before. For that the other slots of the call are looked through.
template <typename E, bool HALF, typename Form>
__device__ __forceinline__ void find_runs(const AppendParams& p, const AppendSide& s, AppendShared& sh) {
  constexpr int kThreads = Form::threads, kHeads = Form::heads;
  const int tid = thread_index(), lane = tid & 31;
  const Share c = share_of<Form>(p);
  const int64_t t0 = c.t0, t1 = c.t1;
  for (int i = tid; i < Form::share * kHeads; i += kThreads) sh.size[i] = 0;
  if (tid < Form::share) sh.first[tid] = INT32_MAX, sh.same[tid] = static_cast<uint8_t>(tid), sh.later[tid] = 0;
  for (int i = tid; i < kMarks / 128; i += kThreads) sh.marks[i] = make_uint4(0, 0, 0, 0);
  if (tid < 32) {
    unsigned long long leads = 0;
    int64_t end = t1, kept = 0;  // tokens of the runs
    int32_t last = t0 > 0 ? block_of(p, slot_of(p, t0 - 1)) : -1;
#pragma unroll
    for (int part = 0; part < Form::share; part += 32) {
      if (t0 + part >= t1) continue;
      const int64_t t = t0 + part + lane;
      const int32_t block = t < t1 ? block_of(p, slot_of(p, t)) : -1;
      const int32_t up = __shfl_up_sync(0xffffffffu, block, 1);
      const bool lead = block >= 0 && (lane == 0 ? last : up) != block;
      const uint32_t bits = __ballot_sync(0xffffffffu, lead), all = __ballot_sync(0xffffffffu, block >= 0);
      if (lead) sh.block[__popcll(leads) + __popc(bits & ((1u << lane) - 1))] = block;
      kept += __popc(leads != 0 ? all : bits != 0 ? all & ~((bits & (0u - bits)) - 1) : 0);
      leads |= static_cast<unsigned long long>(bits) << part;
      last = __shfl_sync(0xffffffffu, block, static_cast<int>(min(t1 - t0 - part, int64_t{32})) - 1);
    }
    while (leads != 0 && last >= 0) {  // the last run may go on behind the share
      const bool on = end + lane < p.T && block_of(p, slot_of(p, end + lane)) == last;
      const uint32_t off = ~__ballot_sync(0xffffffffu, on);
      end += off != 0 ? __ffs(off) - 1 : 32;
      if (off != 0) break;
    }
    // no run has more tokens than its block has places
    const bool parts = kept + (end - t1) != static_cast<int64_t>(__popcll(leads)) * p.block;
    if (lane == 0) sh.leads = leads, sh.end = end, sh.parts = parts, sh.twice = false;
  }
  __syncthreads();
  if (!sh.parts) return;

  const int runs = __popcll(sh.leads), pairs = s.rotated / 2;
  uint32_t* marks = reinterpret_cast<uint32_t*>(sh.marks);
  auto hash_of = [](uint32_t block) { return block * 0x9e3779b1u; };  // bits 17 to 31 are a mark's
  if (tid < runs) {
    const uint32_t h = hash_of(sh.block[tid]), bit = 1u << (h >> 17 & 31);
    if (atomicOr(&marks[h >> 22], bit) & bit) sh.twice = true;
  }
  __syncthreads();
  if (sh.twice && tid < runs)
    for (int r = tid - 1; r >= 0; --r)
      if (sh.block[r] == sh.block[tid]) sh.same[tid] = static_cast<uint8_t>(r);
  // whether a slot's block may be a run's; of a slot that is none, anything
  auto marked = [&](uint32_t slot) -> uint32_t {
    const uint32_t h = hash_of(p.block_shift >= 0 ? slot >> p.block_shift : slot / p.block);
    return __funnelshift_r(marks[h >> 22], 0, h >> 17) & 1;
  };
  const int64_t begin = t0 + __ffsll(static_cast<long long>(sh.leads)) - 1;
  // Tokens that may be of a run's block, one a lane at most: a warp adds up kOnce at a time (one by one
  // 64 sequences' four tokens take 26 us in place of 16).
  auto add = [&](int64_t t, bool may) {
    const int32_t slot = may ? slot_of(p, t) : -1, block = block_of(p, slot);
    int run = -1;
    if (block >= 0)
      for (int r = runs - 1; r >= 0; --r) run = sh.block[r] == block ? r : run;
    if (run >= 0) {
      atomicMin(&sh.first[run], slot - block * p.block);
      if (t < begin) sh.later[run] = 1;
    }
    constexpr int kOnce = 4;
    for (uint32_t which = __ballot_sync(0xffffffffu, run >= 0); which != 0;) {
      const E* token[kOnce];
      int to[kOnce];
#pragma unroll
      for (int i = 0; i < kOnce; ++i) {  // the last one again where there is none
        const int src = which != 0 ? __ffs(which) - 1 : 0;
        to[i] = which != 0 ? __shfl_sync(0xffffffffu, run, src) : to[i > 0 ? i - 1 : 0];
        token[i] = which != 0 ? static_cast<const E*>(s.x) + c.h0 * s.x_head + (t - lane + src) * s.x_token : token[i > 0 ? i - 1 : 0];
        which &= which - 1;
      }
      for (int u = 0; u < c.heads; ++u) {
        float high[kOnce] = {};
#pragma unroll 1
        for (int j = lane; j < s.D - pairs; j += 32) {  // pairs that turn, then elements that do not
          const int n = j - pairs, at = n < 0 ? s.offset + (HALF ? j : 2 * j) : n >= s.offset ? n + s.rotated : n;
          const float factor = n < 0 ? fabsf(p.scale) : 1.0f;
#pragma unroll
          for (int i = 0; i < kOnce; ++i) {
            const E* of = token[i] + u * s.x_head + at;
            const float one = 0.5f * fabsf(Elem<E>::get(of[0]));
            const float two = n < 0 ? 0.5f * fabsf(Elem<E>::get(of[HALF ? pairs : 1])) : 0.0f;
            const float size = (one + two) * factor;
            if (size <= FLT_MAX) high[i] = fmaxf(high[i], size);
          }
        }
#pragma unroll
        for (int i = 0; i < kOnce; ++i) {
          const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(high[i]));
          if (lane == 0) atomicMax(&sh.size[to[i] * kHeads + u], most);
        }
      }
    }
  };
  // What lies before the CTA's tokens, and what behind: kAhead slots a thread at once.
  constexpr int kAhead = 8;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const int64_t to = side == 0 ? begin : p.T;
#pragma unroll 1
    for (int64_t t = (side == 0 ? 0 : sh.end) + tid; t - lane < to; t += kThreads * kAhead) {
      const int32_t* slots = p.slots + t;
      const int left = static_cast<int>(min(to - t, int64_t{kThreads * kAhead}));  // 0 and below: none of this lane's
      uint32_t slot[kAhead], hits = 0;
#pragma unroll
      for (int a = 0; a < kAhead; ++a) slot[a] = a * kThreads < left ? slots[a * kThreads] : 0xffffffffu;
#pragma unroll
      for (int a = 0; a < kAhead; ++a) hits |= marked(slot[a]) << a;
#pragma unroll 1
      for (uint32_t any = __reduce_or_sync(0xffffffffu, hits); any != 0; any &= any - 1) {
        const int a = __ffs(any) - 1;
        add(t + a * kThreads, (hits >> a & 1) != 0 && a * kThreads < left);
      }
    }
  }
  __syncthreads();
}

// One side of a CTA. An item that turns holds two units of V elements: of the first
// half and of the second (HALF), or one behind the other; so does one that does not.
// Without `vector` (V = 2) it holds one pair, or one element.
template <typename E, int V, bool HALF, bool SCALED, typename Form>
__device__ __forceinline__ void append_side(const AppendParams& p, const AppendSide& s, AppendShared& sh) {
  constexpr int kThreads = Form::threads, kRows = Form::rows, kHeads = Form::heads;
  constexpr bool kVector = sizeof(E) * V == 16;
  constexpr int kPairs = kVector ? V : 1;  // of an item
  using VecT = Vec<E, V>;
  const int tid = thread_index(), lane = tid & 31;
  const Share c = share_of<Form>(p);
  const int h0 = c.h0, heads = c.heads;
  const int64_t t0 = c.t0, t1 = c.t1;
  const int per = min(s.items, kThreads);
  const int sub = tid / per, i0 = tid - sub * per, side_by_side = kThreads / per;
  const int sweep = kRows * side_by_side;  // tokens at once
  const int pairs = s.rotated / 2, units = s.rotated / V, rest = (s.D - s.rotated) / V;
  int64_t begin = t0, end = t1;  // of the CTA's tokens

  // ---- an item of a token ----
  const E* x = static_cast<const E*>(s.x) + h0 * s.x_head;
  struct Item {
    bool turns, two;  // it turns pairs; it has a second unit, or a pair's second element
    int at, other;    // of the first and the second in the head
  };
  auto item_of = [&](int i) -> Item {
    auto past = [&](int at) { return at >= s.offset && s.rotated > 0 ? at + s.rotated : at; };
    Item m;
    m.turns = i < s.turn_items;
    if (!kVector) {
      m.two = m.turns;
      m.at = m.turns ? s.offset + i * (HALF ? 1 : 2) : past(i - s.turn_items);
      m.other = m.at + (HALF ? pairs : 1);
    } else if (m.turns && HALF) {
      m.two = true, m.at = s.offset + i * V, m.other = m.at + pairs;
    } else if (m.turns) {
      m.two = 2 * i + 1 < units, m.at = s.offset + 2 * i * V, m.other = m.at + V;
    } else {
      const int u = 2 * (i - s.turn_items);
      m.two = u + 1 < rest, m.at = past(u * V), m.other = past((u + 1) * V);
    }
    return m;
  };
  VecT a[kRows][kHeads], b[kRows][kHeads];  // of an item without a second unit, b is zeros
  int32_t slots[kRows];
  float cosines[kPairs], sines[kPairs];
  auto slots_of = [&](int64_t t) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t at = t + u * side_by_side;
      slots[u] = sub < side_by_side && at < end ? slot_of(p, at) : -1;
    }
  };
  auto load = [&](int64_t t, const Item& m) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (slots[r] < 0) continue;
      const E* from = x + (t + r * side_by_side) * s.x_token;
#pragma unroll
      for (int u = 0; u < kHeads; ++u) {
        if (u >= heads) continue;
        const E* at = from + u * s.x_head;
        if constexpr (kVector) {
          a[r][u] = load16<VecT>(at + m.at);
          if (m.two)
            b[r][u] = load16<VecT>(at + m.other);
          else
            *reinterpret_cast<uint4*>(&b[r][u]) = make_uint4(0, 0, 0, 0);
        } else {
          a[r][u].e[0] = at[m.at];
          if (m.two) a[r][u].e[1] = at[m.other];
        }
      }
    }
  };
  auto angles = [&](int64_t t, int i, const Item& m) {
    if (!m.turns) return;
    const int64_t pos = p.positions_64 ? static_cast<const int64_t*>(p.positions)[t] : static_cast<const int32_t*>(p.positions)[t];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const int pair = i * kPairs + j;
      const uint64_t turn = static_cast<uint64_t>(pos) * sh.rates[pair < pairs ? pair : 0];
      const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
      // 2^-20 by the special function unit (see rotary.cu): 2^-9 of fp16's
      // rounding, 2^-16 of an 8-bit one's; FP32 takes the full functions.
      if constexpr (SCALED || sizeof(E) == 2)
        __sincosf(half_turns * 3.14159265f, &sines[j], &cosines[j]);
      else
        sincospif(half_turns, &sines[j], &cosines[j]);
      cosines[j] *= p.scale, sines[j] *= p.scale;
    }
  };

  // ---- the runs ----
  unsigned long long leads = 0;  // bit per token of the share: it begins a run
  int runs = 0;
  if constexpr (SCALED) {
    leads = sh.leads, end = sh.end;
    if (leads == 0) return;
    runs = __popcll(leads);
    begin = t0 + __ffsll(static_cast<long long>(leads)) - 1;
  }
  // The run of a token between begin and end that is written, the first one of its block.
  auto run_of = [&](int64_t t) -> int { return sh.same[t < t1 ? __popcll(leads & ((2ull << (t - t0)) - 1)) - 1 : runs - 1]; };
  const bool once = end - begin <= sweep && s.items <= kThreads;  // what is loaded stays

  bool odd = false;  // something that this thread holds may not be finite, or not its results
  // Half the largest size of an item of each token, without what is not finite.
  auto sizes_of = [&](const Item& m, uint32_t(&most)[kRows][kHeads]) {
#pragma unroll
    for (int ru = 0; ru < kRows * kHeads; ++ru) {
      const int r = ru / kHeads, u = ru % kHeads;
      if (slots[r] < 0 || u >= heads) continue;
      const VecT &av = a[r][u], &bv = b[r][u];
      float high = 0.0f;
      bool plain = false;
      if constexpr (kVector && sizeof(E) == 2) {
        // the largest number as bits, two at a time: nothing is near the end of FP32's range
        const uint32_t* wa = reinterpret_cast<const uint32_t*>(&av);
        const uint32_t* wb = reinterpret_cast<const uint32_t*>(&bv);
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) bits = max_two(bits, max_two(wa[j] & 0x7fff7fffu, wb[j] & 0x7fff7fffu));
        bits = max(bits & 0xffffu, bits >> 16);
        plain = bits < (std::is_same<E, __half>::value ? 0x7c00u : 0x7e00u);
        if (plain && !m.turns) {
          high = 0.5f * floats_of<E>(bits).x;
        } else if (plain) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 y = floats_of<E>(wa[j]), z = floats_of<E>(wb[j]);
            if (HALF)
              high = fmaxf(high, fmaxf(fmaf(fabsf(y.x), 0.5f, 0.5f * fabsf(z.x)), fmaf(fabsf(y.y), 0.5f, 0.5f * fabsf(z.y))));
            else
              high = fmaxf(high, fmaxf(fmaf(fabsf(y.x), 0.5f, 0.5f * fabsf(y.y)), fmaf(fabsf(z.x), 0.5f, 0.5f * fabsf(z.y))));
          }
          high *= fabsf(p.scale);
          plain = high < 0x1p126f;
        }
      }
      if (!plain) {
        odd = true, high = 0.0f;
        auto count = [&](float size) {
          if (size <= FLT_MAX) high = fmaxf(high, size);
        };
        auto half = [](E e) { return 0.5f * fabsf(Elem<E>::get(e)); };
        if (!kVector) {
          if (m.turns)
            count((half(av.e[0]) + half(av.e[1])) * fabsf(p.scale));
          else
            count(half(av.e[0]));
        } else if (m.turns) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            if (HALF) {
              count((half(av.e[j]) + half(bv.e[j])) * fabsf(p.scale));
            } else if (j % 2 == 0) {
              count((half(av.e[j]) + half(av.e[j + 1])) * fabsf(p.scale));
              count((half(bv.e[j]) + half(bv.e[j + 1])) * fabsf(p.scale));
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) count(half(av.e[j])), count(half(bv.e[j]));
        }
      }
      most[r][u] = max(most[r][u], __float_as_uint(high));
    }
  };

  if constexpr (SCALED) {
    // ---- the largest sizes; a warp's threads stay together ----
    slots_of(begin + sub);
    const Item mine = item_of(i0);
    if (once) load(begin + sub, mine);
    const bool has = tid < runs * kHeads && tid % kHeads < heads && sh.same[tid / kHeads] == tid / kHeads;  // a run and head
    float* scale = s.scales + (has ? static_cast<int64_t>(sh.block[tid / kHeads]) * p.H + h0 + tid % kHeads : 0);
    const float before = has ? *scale : 0.0f;
    for (int64_t from = begin; from < end; from += sweep) {
      if (from > begin) slots_of(from + sub);
      uint32_t most[kRows][kHeads] = {};
      if (once) {
        sizes_of(mine, most);
      } else {
        for (int i = i0; i < s.items; i += per) {
          const Item m = item_of(i);
          load(from + sub, m);
          sizes_of(m, most);
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int run = slots[r] >= 0 ? run_of(from + sub + r * side_by_side) : -1;
        if (run >= 0 && i0 == 0) atomicMin(&sh.first[run], slots[r] - block_of(p, slots[r]) * p.block);
        // one number a warp where it is all of one run (or idle), one a thread otherwise
        const int any = __reduce_max_sync(0xffffffffu, run);
        if (any < 0) continue;
        const bool same = __all_sync(0xffffffffu, run < 0 || run == any);
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
          if (u >= heads) continue;
          if (same) {
            const uint32_t all = __reduce_max_sync(0xffffffffu, most[r][u]);
            if (lane == 0) atomicMax(&sh.size[any * kHeads + u], all);
          } else if (run >= 0) {
            atomicMax(&sh.size[run * kHeads + u], most[r][u]);
          }
        }
      }
    }
    __syncthreads();
    // ---- the scales ----
    if (has) {
      const float need = scale_for(__uint_as_float(sh.size[tid]));
      const bool begins = sh.first[tid / kHeads] == 0, first = sh.later[tid / kHeads] == 0;
      const float now = begins ? need : fmaxf(before, need);  // whether or not another share has written it already
      if (first && (begins || now != before)) *scale = now;
      sh.size[tid] = __float_as_uint(1.0f / now);
      sh.ratio[tid] = begins || !first ? 1.0f : before / now;
    } else if (tid < runs * kHeads) {
      sh.ratio[tid] = 1.0f;
    }
    __syncthreads();
  }

  // ---- the tokens ----
  for (int64_t from = begin; from < end; from += sweep) {
    const int64_t t = from + sub;
    if (!SCALED || !once) slots_of(t);
    for (int i = i0; i < s.items; i += per) {
      const Item m = item_of(i);
      if (!SCALED || !once) load(t, m);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int32_t slot = slots[r];
        if (slot < 0) continue;
        const int32_t page = p.page_shift >= 0 ? slot >> p.page_shift : slot / p.page_size;
        const int64_t entry = page * s.page + (slot - page * p.page_size) * s.entry + h0 * s.head;
        const int run = SCALED ? run_of(t + r * side_by_side) : 0;
        angles(t + r * side_by_side, i, m);
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
          if (u >= heads) continue;
          const VecT &av = a[r][u], &bv = b[r][u];
          // the item's elements, two at a time, of the second unit in z
          constexpr int kTwos = V / 2;
          uint64_t y[kTwos], z[kTwos];
          if constexpr (kVector) {
#pragma unroll
            for (int j = 0; j < kTwos; ++j) {
              y[j] = pair(Elem<E>::get(av.e[2 * j]), Elem<E>::get(av.e[2 * j + 1]));
              z[j] = pair(Elem<E>::get(bv.e[2 * j]), Elem<E>::get(bv.e[2 * j + 1]));
            }
          } else {
            y[0] = pair(Elem<E>::get(av.e[0]), m.two ? Elem<E>::get(av.e[1]) : 0.0f), z[0] = 0;
          }
          if (m.turns) {
            if constexpr (kVector && HALF) {
#pragma unroll
              for (int j = 0; j < kTwos; ++j) {
                const uint64_t c = pair(cosines[2 * j], cosines[2 * j + 1]), d = pair(sines[2 * j], sines[2 * j + 1]);
                const uint64_t first = fma2(y[j], c, mul2(z[j], pair(-sines[2 * j], -sines[2 * j + 1])));
                z[j] = fma2(z[j], c, mul2(y[j], d));
                y[j] = first;
              }
            } else {
              auto turn = [&](uint64_t& v, int j) {
                const float2 w = both(v);
                v = pair(w.x * cosines[j] - w.y * sines[j], w.y * cosines[j] + w.x * sines[j]);
              };
#pragma unroll
              for (int j = 0; j < kTwos; ++j) {
                turn(y[j], j);
                if constexpr (kVector) turn(z[j], kTwos + j);
              }
            }
          }
          if constexpr (SCALED) {
            uint8_t* to = static_cast<uint8_t*>(s.cache) + entry + u * s.head;
            const uint64_t unit = twice(__uint_as_float(sh.size[run * kHeads + u]));
            if (!once || odd) {  // a product with 0 is 0, or NaN of what is not finite
#pragma unroll
              for (int j = 0; j < kTwos; ++j) y[j] = fma2(y[j], 0, y[j]), z[j] = fma2(z[j], 0, z[j]);
            }
            auto two = [&](uint64_t v) -> uint32_t {
              const float2 w = both(mul2(v, unit));
              return e4m3_two(w.x, w.y);
            };
            if constexpr (kVector) {
              auto put = [&](uint8_t* to, const uint64_t(&y)[kTwos]) {
                uint32_t w[V / 4];
#pragma unroll
                for (int j = 0; j < V / 4; ++j) w[j] = two(y[2 * j]) | two(y[2 * j + 1]) << 16;
                if constexpr (V == 8)
                  *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
                else
                  *reinterpret_cast<uint32_t*>(to) = w[0];
              };
              put(to + m.at, y);
              if (m.two) put(to + m.other, z);
            } else {
              const uint32_t w = two(y[0]);
              to[m.at] = static_cast<uint8_t>(w);
              if (m.two) to[m.other] = static_cast<uint8_t>(w >> 8);
            }
          } else {
            E* to = static_cast<E*>(s.cache) + entry + u * s.head;
            VecT c;
            auto pack = [&](const uint64_t(&y)[kTwos]) {
#pragma unroll
              for (int j = 0; j < kTwos; ++j) {
                const float2 w = both(y[j]);
                c.e[2 * j] = Elem<E>::put(w.x), c.e[2 * j + 1] = Elem<E>::put(w.y);
              }
            };
            pack(y);
            if constexpr (kVector) {
              store16(to + m.at, c);
              if (m.two) pack(z), store16(to + m.other, c);
            } else {
              to[m.at] = c.e[0];
              if (m.two) to[m.other] = c.e[1];
            }
          }
        }
      }
    }
  }

  if constexpr (SCALED) {
    // ---- earlier entries of blocks whose scale grew, one run and head a warp ----
    for (int j = tid >> 5; j < runs * kHeads; j += kThreads / 32) {
      const int r = j / kHeads, u = j % kHeads;
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

template <typename E, bool HALF, bool SCALED, typename Form>
__global__ void __launch_bounds__(Form::threads, Form::per_sm) append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ AppendShared sh;
  const AppendSide& s = p.side[blockIdx.y];
  for (int i = threadIdx.x; i < s.rotated / 2; i += Form::threads) sh.rates[i] = turns_of(p.frequencies[i]);
  if constexpr (SCALED)
    find_runs<E, HALF, Form>(p, s, sh);
  else
    __syncthreads();
  if (s.vector)
    append_side<E, 16 / sizeof(E), HALF, SCALED, Form>(p, s, sh);
  else
    append_side<E, 2, HALF, SCALED, Form>(p, s, sh);
}

bool aligned_to(const void* q, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(q) & (bytes - 1)) == 0; }

// Many tokens: a block of 64 with heads of 128 stays in a CTA's registers (8192 tokens
// x 8 heads x (128 + 128), bf16, into 8 bits: 34 us by two heads a thread and three CTAs
// an SM, 40 by two CTAs, 39 by four heads; into 16 bits, which wait on nothing between,
// 12.3 for 10.4 by four heads). Few: small CTAs, so that all SMs have some (64 tokens
// 8.4 us, 14.6 by large ones).
using ScaledForm = FormOf<256, 2, 2, 3, 64>;
using PlainForm = FormOf<256, 2, 4, 2, 64>;
using FewForm = FormOf<128, 1, 1, 4, 16>;

template <typename E, bool HALF, bool SCALED, typename Form>
topk_status launch_form(const AppendParams& p, int sides, int sm_count, cudaStream_t stream) {
  AppendParams q = p;
  q.head_groups = (p.H + Form::heads - 1) / Form::heads;
  auto grid_of = [&](int share) { return (static_cast<int64_t>(p.T) + share - 1) / share * q.head_groups; };
  q.share = Form::share;
  while (q.share > 1 && grid_of(q.share) * sides < 2 * sm_count) q.share /= 2;
  const int64_t grid = grid_of(q.share);
  if (grid > INT32_MAX) return TOPK_EINVAL;
  const dim3 g(static_cast<unsigned>(grid), static_cast<unsigned>(sides));
  return launch(append_kernel<E, HALF, SCALED, Form>, q, g, Form::threads, 0, stream);
}

template <typename E, bool HALF, bool SCALED>
topk_status launch_layout(const AppendParams& p, int sides, int sm_count, cudaStream_t stream) {
  double items = 0.0;
  for (int i = 0; i < sides; ++i) items += p.side[i].items;
  // with four CTAs of 256 threads to each SM
  if (items * p.T * p.H >= 1024.0 * sm_count)
    return launch_form<E, HALF, SCALED, std::conditional_t<SCALED, ScaledForm, PlainForm>>(p, sides, sm_count, stream);
  return launch_form<E, HALF, SCALED, FewForm>(p, sides, sm_count, stream);
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
  p.page_shift = p.block_shift = -1;
  for (int i = 0; i < 31; ++i) {
    if (p.page_size == 1 << i) p.page_shift = i;
    if (p.block == 1 << i) p.block_shift = i;
  }
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
    // two units an item
    s.turn_items = s.vector ? (s.rotated / V + 1) / 2 : s.rotated / 2;
    s.items = s.turn_items + (s.vector ? ((s.D - s.rotated) / V + 1) / 2 : s.D - s.rotated);
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
