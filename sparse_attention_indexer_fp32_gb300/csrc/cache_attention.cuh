// Attention over selected entries of a paged cache in 8 bits
// (include/sparse_cache.h, sparse_attention_e4m3).
//
// The products. Entries go from the cache into the tensor cores as they are, in
// E4M3, with no conversion on the way: kind f8f6f4 takes both operands in 8 bits,
// so queries and weights are split into E4M3 terms, x = u (t0 + t1 / 16 + t2 / 256),
// each the rounded rest of those before. A term adds five bits (four and the
// rest's sign): two hold 9, a bf16 query exactly; three hold 14, an fp16 query
// exactly. Two terms of a weight round it to 2^-9 of itself, half of what bf16 would;
// three are good to fp16's 2^-11, which it is rounded to first. A query's unit u is
// a power of two, its head's own.
//
// The tile. 128 entries are the rows of both products and their (term, head) pairs
// the columns: S = K Q^T, and O^T += V^T P with P read along the entries. So few
// heads a key head cost few columns instead of empty rows, each term has sums of
// its own, joined with their factors in FP32 registers, and one thread has one
// entry: its scales, mask and position are scalars, and every exponential is one
// thread's own.
//
// The scales. A key's scale multiplies its logit. A value's multiplies its weight
// before that is split: w = 2^(z - r) s. The reference r of a head is moved, for
// all threads at once, when a weight would pass E4M3's 448, to leave the largest in
// (2^6, 2^7]. The last term ends at steps of 2^-13 (three terms: 2^-17), 2^-19 (2^-23) of
// the largest weight there is. The
// sum that divides adds the weights in FP32, unrounded and without the values' scales. r
// is a whole number, so moving it is exact but for logits that were rounded next to the
// old one: past kFar those are computed anew. Whether a head's reference moves in a tile, and
// by how much, follows from its own logits and the CTA's tiles. Its last bits follow from
// more: from how many CTAs share a row, which the call's works decide, and from the other
// heads of its set, where one of them passes kFar and all logits are rounded once, not twice.
//
// The rest is as in sparse_attention.cu: entries gathered by 16-byte copies into
// rings of keys and values, few rows shared by a cluster whose CTAs join through
// distributed shared memory, CTAs that stay for several rows where there are many.
//
// Warps: 4 softmax warps for each 16 heads (G = 8: for all 8), one entry a thread;
// 4 or 8 that gather; one thread issues all products; 3 or 7 split queries ahead. Softmax
// warps take registers from the others (setmaxnreg; 88 instead of 72 with 64 heads: a tile
// that moves a reference spilled them, 182 us against 150 below).
//
// Bounds. Few heads and long lists: the entries' bytes. Many heads: the softmax warps (a
// logit's two terms joined, scaled, an exponential, a sum, two roundings to E4M3 and the
// rest between them: with loads and gathers thirty instructions), and a row's end, where they wait for the last product,
// sum and write while the tensor cores wait for them: there is one set of sums, though TMEM
// would hold a second one but for values past 128 with 64 heads (fp16: 32, and 16 with two CTAs
// an SM); and a moved reference, for which a set waits for the product before.
// Figures, in a CUDA graph:
//   2048 rows x 64 heads over 512 shared entries of 256: 166 us, 32 of them at the rate of
//   bf16 products (135 where no reference moves; 270 over 1024 entries, 80 over 128; 32 heads
//   130, 16 heads 91, 8 heads 64, there 4.2 TB/s of entries out of L2). 62 thousand warp
//   instructions a row, some 7.6 of them a tile that moves nothing; issue slots 70 %. In fp16 268,
//   141, 103 and 70 us for 64, 32, 16 and 8 heads;
//   64 rows x 8 x 8 heads of 128 over 2048 entries: 59 us, 6 TB/s less a start of some 12 us
//   (launch, list, page, entries, one behind the other); 4 rows over 512 entries 12.1 us.
// Lost, against 147 to 150 us with references that moved less: dedicated warps that read the sums out (226 us: registers), two CTAs an SM with tiles
// of 32 heads for 64 (270: entries are read twice), all columns of a set multiplied where one
// reference moves (179), results by way of shared memory (32 heads 129 for 123).
#include <cuda_runtime.h>

#include <cfloat>
#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "attention_math.cuh"
#include "cache_launch.cuh"
#include "e4m3.cuh"
#include "step_launch.cuh"
#include "tcgen05.cuh"

namespace tki {
namespace {

constexpr int kEntries = 128;  // of a tile
constexpr int kMaxStages = 6;
constexpr int kBufs = 2;  // buffers of scores in TMEM, of weights and queries in shared memory
constexpr int kMaxNotes = kMaxStages + kBufs;  // see E4Params::notes
constexpr float kNoHead = 1073741824.0f;  // the reference of heads that are none: no weight
constexpr float kLogLimit = 8.8073549f;     // log2(448)
// A reference leaves the largest weight in (2^(kTop - 1), 2^kTop] when it is set, so that it seldom
// moves again and the last term's steps are 2^-19 (2^-23) of that weight at most: half a step of each
// of 2048 entries is a quarter of a step of bf16 (an eighth of fp16's) together. 64 heads on 512 shared entries 167 us;
// 146 by (2^3, 2^4], steps of 2^-16, with which the rest beside one large weight loses its digits.
constexpr float kTop = 7.0f;
constexpr int kLongest = 2048;  // entries of one reference; CTAs share longer lists, up to eight
constexpr float kFar = 16.0f;  // a reference that moves further has left logits with less than 2^-20 of their digits
constexpr float kLeast = 0x1p-60f;          // values' scales below count as this for the reference

template <typename E, int G>
struct Shape {
  static constexpr int terms = std::is_same<E, __nv_bfloat16>::value ? 2 : 3;
  static constexpr int set_heads = G < 16 ? G : 16;  // of one set of four softmax warps
  static constexpr int sets = G / set_heads;
  static constexpr int rows = terms * G;           // (term, head) pairs
  static constexpr int N = (rows + 15) / 16 * 16;  // columns; those past the rows hold nothing
  static constexpr int p_bytes = N * kEntries;     // of a buffer of weights
  static constexpr int softmax = 4 * sets, gather = G <= 32 ? 8 : 4, queries = G <= 16 ? 3 : 7;  // warps
  static constexpr int mma = softmax + gather, query = mma + 1;
  static constexpr int threads = (query + queries) * 32;
  static constexpr int per_sm = G <= 16 ? 2 : 1;
  // Registers a thread: at the launch, and of the groups of four warps of each kind. Gathering
  // wants 64 where entries are few heads' (64 x 8 x 8 heads 57 us, 59.6 with 56 and 96 for softmax);
  // with 64 heads softmax wants them (150 us, 156 with 80, 56 and 56, when references moved less), then
  // gathering (137 us without a moved reference, 142 with 48).
  static constexpr int regs = G <= 16 ? 64 : G == 32 ? 80 : 72;
  static constexpr int softmax_regs = G <= 16 ? 80 : G == 32 ? 120 : 88;
  static constexpr int gather_regs = G <= 32 ? 64 : 56, query_regs = G == 32 ? 56 : 48;
  static_assert(softmax % 4 == 0 && gather % 4 == 0 && (queries + 1) % 4 == 0);
  static_assert(softmax * softmax_regs + gather * gather_regs + (queries + 1) * query_regs <= (threads / 32) * regs);
};

// The registers of each thread of four warps.
template <int FROM, int TO>
__device__ __forceinline__ void registers() {
  if constexpr (TO > FROM)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TO));
  else if constexpr (TO < FROM)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TO));
}

struct E4Params {
  sparse_attention_args a;
  const float* k_scales;
  const float* v_scales;
  int32_t block, blocks;   // entries of a block, blocks a page
  int32_t heads, h_tiles;  // query heads per key head, tiles of G of them
  uint32_t works;          // (row, key head, tile of heads)
  int32_t d_blocks, v_blocks, d_steps;  // 128-byte blocks of an entry, 32-byte steps of its keys
  int32_t shared;                       // v is a prefix of k's entries
  int32_t page_shift, block_shift;      // log2, or -1
  uint32_t pages, table_width;
  int32_t k_stages, v_stages, k_bytes, v_bytes;
  // What is noted of each entry (scales, distance, mask) outlives its keys' stage:
  // S of tile i follows the softmax of tile i - kBufs, so tile i's notes may go where
  // those of tile i - k_stages - kBufs were once S of tile i - k_stages is there.
  int32_t notes;
  int32_t k_at, v_at, p_at, note_at, shared_at;  // in shared memory, after Q
  int32_t note_bytes;
  int32_t tmem_cols;
  float scale_log2e, scale_over_cap, cap_log2e;
  bool q_vector;
};

// Of a tile's entries; `away` only with slopes.
struct Notes {
  float ks[kEntries], vs[kEntries];
  uint32_t seen[4];
  float away[kEntries];
};

template <int G, int SETS, int HS>
struct E4Shared {
  alignas(16) float nref[G];  // a head's reference, negative; +0: nothing seen yet, a reference of 0 is -0
  alignas(16) float step[G];  // what was last added to nref, and the factor of its sums
  alignas(16) float factor[G];
  alignas(16) float inverse[G];
  alignas(16) float unit[4][G];  // of the queries, of the last four works
  float most[SETS * 4][HS], sum[SETS * 4][HS];
  float head_ref[G], head_sum[G];  // for the other CTAs of a cluster
  uint64_t k_full[kMaxStages], v_full[kMaxStages];
  uint64_t q_full[kBufs], q_empty[kBufs], units[4];
  // Of tile i at i % 8: scores there, weights there, products with v done.
  uint64_t s_full[8], p_full[8], pv_done[8];
  uint64_t drained;
  uint32_t tmem;
  uint32_t stop;
};

struct E4Work {
  int g, heads, head0;  // key head; real heads, and the first one's query head
  int64_t row, b, t;
};

template <int G>
__device__ __forceinline__ E4Work e4_work(const E4Params& p, uint32_t w) {
  E4Work r;
  const uint32_t pair = w / static_cast<uint32_t>(p.h_tiles), row = pair / static_cast<uint32_t>(p.a.Hkv);
  const int tile = static_cast<int>(w - pair * p.h_tiles);
  const uint32_t b = row / static_cast<uint32_t>(p.a.T);
  r.g = static_cast<int>(pair - row * p.a.Hkv);
  r.heads = min(p.heads - tile * G, G);
  r.head0 = r.g * p.heads + tile * G;
  r.row = row, r.b = b, r.t = row - b * static_cast<uint32_t>(p.a.T);
  return r;
}

__device__ __forceinline__ void put16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Among the 128 threads of a set: whether any of them says yes.
__device__ __forceinline__ bool set_any(int set, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, %2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(yes ? 1u : 0u), "r"(set + 1)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void set_sync(int set) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(set + 1) : "memory"); }

// Sums of HS numbers over the lanes of a warp: lane l is left with that of number
// l / (32 / HS).
template <int HS>
__device__ __forceinline__ float sum_lanes(float (&v)[HS], int lane) {
#pragma unroll
  for (int w = HS / 2, bit = 16; w >= 1; w /= 2, bit /= 2) {
    const bool high = lane & bit;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float give = high ? v[i] : v[i + w], keep = high ? v[i + w] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
    }
  }
#pragma unroll
  for (int bit = 32 / HS / 2; bit >= 1; bit /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
  return v[0];
}

// The same for the largest.
template <int HS>
__device__ __forceinline__ float max_lanes(float (&v)[HS], int lane) {
#pragma unroll
  for (int w = HS / 2, bit = 16; w >= 1; w /= 2, bit /= 2) {
    const bool high = lane & bit;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float give = high ? v[i] : v[i + w], keep = high ? v[i + w] : v[i];
      v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, bit));
    }
  }
#pragma unroll
  for (int bit = 32 / HS / 2; bit >= 1; bit /= 2) v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], bit));
  return v[0];
}

// The two numbers of 32 bits of queries.
template <typename E>
struct Two;
template <>
struct Two<__nv_bfloat16> {
  static __device__ __forceinline__ float2 get(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
};
template <>
struct Two<__half> {
  static __device__ __forceinline__ float2 get(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
};

__device__ __forceinline__ float log2_fast(float x) {  // to 2^-22 of 1 or of itself
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half_two(float x, float y) {
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t e4m3_of_half2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
// 16 (x - y), exact where y is a term of x.
__device__ __forceinline__ uint32_t rest16(uint32_t x, uint32_t y) {
  const __half2 a = *reinterpret_cast<const __half2*>(&x), b = *reinterpret_cast<const __half2*>(&y);
  const __half2 r = __hmul2(__hsub2(a, b), __float2half2_rn(16.0f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Descriptor of the weights: units of 16 (term, head) pairs, one behind the other, entry e
// of a unit at byte e * 16 of it. Not swizzled: a thread writes whole units, its neighbours
// the next ones.
__device__ __forceinline__ uint64_t weights_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (static_cast<uint64_t>((8 * 16) >> 4) << 16) |
         (static_cast<uint64_t>((kEntries * 16) >> 4) << 32) | (1ull << 46);
}

// Whether a negative reference is still that of a head that has seen nothing.
__device__ __forceinline__ bool begins(float nref) { return __float_as_uint(nref) == 0; }

// 1 / a sum of weights, zero where nothing is seen; and its logarithm with the reference.
__device__ __forceinline__ float e4_inverse(float sum) { return sum == 0.0f ? 0.0f : reciprocal(sum); }
__device__ __forceinline__ float e4_logsum(float ref, float sum) {
  return sum != sum ? sum : sum == 0.0f ? __int_as_float(0xff800000) : (ref + log2f(sum)) * kLn2;
}

template <typename E, int G>
__global__ void __launch_bounds__(Shape<E, G>::threads, Shape<E, G>::per_sm)
    cache_attention_kernel(const __grid_constant__ E4Params p, const int cluster) {
  extern __shared__ __align__(1024) unsigned char smem[];
  using S = Shape<E, G>;
  constexpr int TERMS = S::terms, HS = S::set_heads, SETS = S::sets, N = S::N;
  using Shared = E4Shared<G, SETS, HS>;
  Shared& sh = *reinterpret_cast<Shared*>(smem + p.shared_at);
  const sparse_attention_args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster > 1 ? cluster_ctarank() : 0;
  const uint32_t step_w = gridDim.x / cluster, first_w = blockIdx.x / cluster;
  const int all_tiles = a.K / kEntries + (a.K % kEntries != 0);
  const int tiles = all_tiles > static_cast<int>(rank) ? (all_tiles - static_cast<int>(rank) + cluster - 1) / cluster : 0;
  const uint32_t base = smem_addr(smem);
  const uint32_t k_ring = base + p.k_at, v_ring = base + p.v_at, p_at = base + p.p_at;
  const int q_block = S::rows * 128, q_bytes = q_block * p.d_blocks;
  constexpr int kSets = S::gather / 4;  // of gathering warps, which take tiles in turn

  // A gathering warp has 32 entries of every tile of its set, one a lane to look up: in the
  // list two of the set's tiles ahead, in the page table one; the first before anything else.
  const bool gathers = warp >= S::softmax && warp < S::mma;
  const int part = (warp - S::softmax) & 3, turn = (warp - S::softmax) >> 2;
  const bool some = a.page_size > 0 && a.num_pages > 0;
  struct Look {
    const int32_t* indices;
    const int32_t* table;
    int32_t last, first, g;
  };
  auto enter = [&](uint32_t w_at) -> Look {
    const E4Work k = e4_work<G>(p, w_at);
    Look l;
    l.indices = a.indices + k.row * a.K;
    l.table = a.page_table != nullptr ? a.page_table + k.b * a.table_stride : nullptr;
    l.last = a.query_positions != nullptr ? a.query_positions[k.row] : INT32_MAX;
    l.first = a.first != nullptr ? max(a.first[k.row], 0) : 0;
    l.g = k.g;
    return l;
  };
  // Tiles are taken from the list's last to its first: a selection comes in ascending order,
  // and with a distance bias the nearest entries have the largest logits.
  auto index_of = [&](const Look& l, int i) -> int32_t {
    const int64_t j = (all_tiles - 1 - (static_cast<int64_t>(i) * cluster + rank)) * kEntries + part * 32 + lane;
    return i < tiles && j < a.K && some ? l.indices[j] : -1;
  };
  auto page_index = [&](int32_t pos) -> uint32_t {
    return p.page_shift >= 0 ? static_cast<uint32_t>(pos) >> p.page_shift
                             : static_cast<uint32_t>(pos) / static_cast<uint32_t>(a.page_size);
  };
  auto page_of = [&](const Look& l, int32_t pos) -> uint32_t {  // ~0: not seen
    if (pos < l.first || pos > l.last) return 0xffffffffu;
    const uint32_t page = page_index(pos);
    return l.table == nullptr ? page : page < p.table_width ? static_cast<uint32_t>(l.table[page]) : 0xffffffffu;
  };
  Look look = {};
  int32_t pos = -1, pos1 = -1;
  uint32_t page = 0xffffffffu;
  if (gathers) look = enter(first_w), pos = index_of(look, turn), pos1 = index_of(look, turn + kSets);

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.k_stages; ++i) mbar_init(&sh.k_full[i], 128 + 4);
    for (int i = 0; i < p.v_stages; ++i) mbar_init(&sh.v_full[i], 128);
    for (int i = 0; i < kBufs; ++i) mbar_init(&sh.q_full[i], S::queries), mbar_init(&sh.q_empty[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&sh.units[i], S::queries);
    for (int i = 0; i < 8; ++i)
      mbar_init(&sh.s_full[i], 2), mbar_init(&sh.p_full[i], S::softmax), mbar_init(&sh.pv_done[i], 1);
    mbar_init(&sh.drained, 1);
    sh.stop = 0;
    fence_mbar_init();
  }
  if (warp == S::mma) tmem_alloc(&sh.tmem, p.tmem_cols);
  if (gathers) page = page_of(look, pos);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_s = sh.tmem, tmem_o = tmem_s + kBufs * N;
  volatile uint32_t* stop = &sh.stop;
  bool one = false;  // the thread that issues products

  if (gathers) {
    // ---- gather ----
    registers<S::regs, S::gather_regs>();
    // 16-byte units of an entry's keys: those that it has, and those that are read
    const int k_units = a.D / 16, k_read = p.d_steps * 2, v_units = a.Dv / 16;
    const uint32_t unit16 = lane & 7, sub = lane >> 3;
    const uint32_t at = (part * 32 + sub) * 128;
    const uint32_t even = (unit16 ^ sub) << 4, odd = (unit16 ^ (sub + 4)) << 4;
    // an empty cache has no address: nothing is read from the one it gets
    const char* nowhere = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(a.q) & ~static_cast<uintptr_t>(15));
    bool ok = true;
    int k_stage = turn % p.k_stages, v_stage = p.shared ? 0 : turn % p.v_stages, note = turn;
    int before_w = 0;  // tiles of the works before
    for (uint32_t w_at = first_w; w_at < p.works && ok; w_at += step_w, before_w += tiles) {
      const int i0 = (turn - before_w) & (kSets - 1), next_i0 = (turn - before_w - tiles) & (kSets - 1);
      const char* keys = some ? static_cast<const char*>(a.k) + look.g * a.k_head_stride + unit16 * 16 : nowhere;
      const char* values = some ? static_cast<const char*>(a.v) + look.g * a.v_head_stride + unit16 * 16 : nowhere;
      // the next work's first entries
      Look next = look;
      int32_t next_pos = -1, next_pos1 = -1;
      uint32_t next_page = 0xffffffffu;
      const bool more = w_at + step_w < p.works;
      if (more) next = enter(w_at + step_w), next_pos = index_of(next, next_i0), next_pos1 = index_of(next, next_i0 + kSets);
      for (int i = i0; i < tiles; i += kSets) {
        const int n = before_w + i;  // the tile's number in the CTA
        const int32_t pos2 = index_of(look, i + 2 * kSets);
        const uint32_t page1 = page_of(look, pos1);
        const bool seen = page < p.pages;
        const uint32_t place = static_cast<uint32_t>(pos) - page_index(pos) * static_cast<uint32_t>(a.page_size);
        const uint32_t bits = __ballot_sync(0xffffffffu, seen);
        // 8 lanes fetch 128 bytes of an entry; step j has entries 4 j + lane / 8. What is not
        // seen is zeros; of a last block that is not full, the units up to `read`.
        auto fetch = [&](uint32_t dst, const char* from, int64_t entry, int units, int read) {
          const int u = static_cast<int>(unit16);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const char* row = from + __shfl_sync(0xffffffffu, entry, 4 * j + sub);
            const uint32_t bytes = (bits >> (4 * j + sub)) & 1 ? 16 : 0, to = dst + j * 512 + (j & 1 ? odd : even);
            if (u < read) copy_bytes(to, row, u < units ? bytes : 0);
            if (u + 8 < read) copy_bytes(to + kEntries * 128, row + 128, u + 8 < units ? bytes : 0);
          }
        };
        int before = n - p.k_stages;
        uint64_t* used = p.shared ? sh.pv_done : sh.s_full;  // when a stage of keys is free
        ok = before < 0 || wait_or_stop(&used[before & 7], (before >> 3) & 1, stop);
        if (!ok) break;
        fetch(k_ring + k_stage * p.k_bytes + at, keys, seen ? page * a.k_page_stride + place * a.k_token_stride : 0,
              k_units, k_read);
        Notes& notes = *reinterpret_cast<Notes*>(smem + p.note_at + note * p.note_bytes);
        const int e = part * 32 + lane;
        const uint32_t block = p.block_shift >= 0 ? place >> p.block_shift : place / static_cast<uint32_t>(p.block);
        const int64_t unit = seen ? (static_cast<int64_t>(page) * p.blocks + block) * a.Hkv + look.g : 0;
        copy4(smem_addr(&notes.ks[e]), some ? reinterpret_cast<const char*>(p.k_scales + unit) : nowhere, seen);
        copy4(smem_addr(&notes.vs[e]), some ? reinterpret_cast<const char*>(p.v_scales + unit) : nowhere, seen);
        copy_arrive(&sh.k_full[k_stage]);
        if (a.slopes != nullptr) notes.away[e] = static_cast<float>(seen ? pos - look.last : 0);
        if (lane == 0) notes.seen[part] = bits;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.k_full[k_stage]);
        if (!p.shared) {
          before = n - p.v_stages;
          ok = before < 0 || wait_or_stop(&sh.pv_done[before & 7], (before >> 3) & 1, stop);
          if (!ok) break;
          fetch(v_ring + v_stage * p.v_bytes + at, values, seen ? page * a.v_page_stride + place * a.v_token_stride : 0,
                v_units, v_units);
          copy_arrive(&sh.v_full[v_stage]);
          v_stage += kSets;
          while (v_stage >= p.v_stages) v_stage -= p.v_stages;
        }
        pos = pos1, pos1 = pos2, page = page1;
        k_stage += kSets, note += kSets;
        while (k_stage >= p.k_stages) k_stage -= p.k_stages;
        if (note >= p.notes) note -= p.notes;
        if (i + 2 * kSets >= tiles && i + kSets < tiles && more) next_page = page_of(next, next_pos);
      }
      if (more && i0 + kSets >= tiles) next_page = page_of(next, next_pos);
      look = next, pos = next_pos, pos1 = next_pos1, page = next_page;
    }
    copy_commit();
    copy_wait<0>();
    registers<S::gather_regs, S::regs>();
  } else if (warp >= S::mma) {
    registers<S::regs, S::query_regs>();  // one instruction for the four warps of a group
    if (warp == S::mma) {
      // ---- products, all by one thread: S of the next tile, then O^T of this one ----
      // So scores that are there say that the weights of the tile two before were used, and
      // a work's first weights that the sums of the one before have been read.
      one = elect_one();
      if (tiles > 0 && one) {
        const uint32_t s_desc = mma_desc(0, N), o_desc = mma_desc(0, N, true, true);
        const uint64_t q_desc = operand_desc(base), k_desc = operand_desc(k_ring);
        const uint64_t v_desc = operand_desc(p.shared ? k_ring : v_ring), p_desc = weights_desc(p_at);
        const int v_stages = p.shared ? p.k_stages : p.v_stages, v_bytes = p.shared ? p.k_bytes : p.v_bytes;
        const int last = static_cast<int>((p.works - first_w + step_w - 1) / step_w) * tiles;  // first_w < works
        int k_stage = 0, k_turn = 0, v_stage = 0, v_turn = 0;
        int s_work = 0, s_tile = 0, o_tile = 0;
        bool ok = true;
        auto scores = [&](int n) {
          const int qb = s_work & 1;
          if (s_tile == 0) ok = wait_or_stop_one(&sh.q_full[qb], (s_work >> 1) & 1, stop);
          ok = ok && wait_or_stop_one(&sh.k_full[k_stage], k_turn, stop);
          if (!ok) return;
          fence_proxy_async_smem();
          tc_fence_after();
          const uint64_t kd = k_desc + static_cast<uint32_t>(k_stage * p.k_bytes >> 4);
          const uint64_t qd = q_desc + static_cast<uint32_t>(qb * q_bytes >> 4);
          const uint32_t to = tmem_s + (n & 1) * N;
          for (int j = 0; j < p.d_steps; ++j) {
            const uint32_t c = j >> 2, in = (j & 3) * 2;
            mma_f8(to, kd + (c * (kEntries * 128 >> 4) + in), qd + (c * (S::rows * 128 >> 4) + in), s_desc, j > 0);
          }
          mma_commit(&sh.s_full[n & 7]);
          mbar_arrive(&sh.s_full[n & 7]);  // by this thread, which has seen the tile's notes
          if (++k_stage == p.k_stages) k_stage = 0, k_turn ^= 1;
          if (++s_tile == tiles) {
            mma_commit(&sh.q_empty[qb]);
            s_tile = 0, ++s_work;
          }
        };
        scores(0);
        for (int n = 0; n < last && ok; ++n) {
          if (n + 1 < last) scores(n + 1);
          if (!p.shared) ok = ok && wait_or_stop_one(&sh.v_full[v_stage], v_turn, stop);
          ok = ok && wait_or_stop_one(&sh.p_full[n & 7], (n >> 3) & 1, stop);
          if (!ok) break;
          fence_proxy_async_smem();
          tc_fence_after();
          const uint64_t vd = v_desc + static_cast<uint32_t>(v_stage * v_bytes >> 4);
          const uint64_t pd = p_desc + static_cast<uint32_t>((n & 1) * S::p_bytes >> 4);
          for (int m = 0; m < p.v_blocks; ++m)
#pragma unroll
            for (int j = 0; j < kEntries / 32; ++j)
              mma_f8(tmem_o + m * N, vd + static_cast<uint32_t>((m * (kEntries * 128) + j * (32 * 128)) >> 4),
                     pd + static_cast<uint32_t>(j * (32 * 16) >> 4), o_desc, o_tile + j > 0);
          mma_commit(&sh.pv_done[n & 7]);
          if (++v_stage == v_stages) v_stage = 0, v_turn ^= 1;
          if (++o_tile == tiles) o_tile = 0;
        }
      }
      __syncwarp();
    } else {
      // ---- queries: a power of two for each head and terms in units of it ----
      // A warp has every so many heads, kAhead of them at once; the next ones, of this work or
      // the next, are on their way meanwhile.
      const int who = warp - S::query;
      constexpr int kAhead = 2;
      uint4 raw[kAhead];
      auto load = [&](const E4Work& k, int h0) {
        const E* q = static_cast<const E*>(a.q) + k.b * a.q_seq_stride + k.t * a.q_token_stride + k.head0 * a.q_head_stride;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int h = h0 + u * S::queries;
          const E* from = q + h * a.q_head_stride + lane * 8;
          raw[u] = make_uint4(0, 0, 0, 0);
          if (h >= k.heads || lane * 8 >= a.D) continue;  // D is a multiple of 16
          if (p.q_vector) {
            raw[u] = *reinterpret_cast<const uint4*>(from);
          } else {
            const uint16_t* e = reinterpret_cast<const uint16_t*>(from);
            auto two = [&](int j) { return e[j] | static_cast<uint32_t>(e[j + 1]) << 16; };
            raw[u] = make_uint4(two(0), two(2), two(4), two(6));
          }
        }
      };
      int nw = 0;
      E4Work k = e4_work<G>(p, first_w);
      if (tiles > 0) load(k, who);
      for (uint32_t w_at = first_w; tiles > 0 && w_at < p.works; w_at += step_w, ++nw) {
        const int qb = nw & 1, heads = k.heads;
        if (nw >= kBufs && !wait_or_stop(&sh.q_empty[qb], ((nw >> 1) - 1) & 1, stop)) break;
        unsigned char* to = smem + qb * q_bytes;
        for (int h0 = who; h0 < G; h0 += S::queries * kAhead) {
          uint4 now[kAhead];
#pragma unroll
          for (int u = 0; u < kAhead; ++u) now[u] = raw[u];
          if (h0 + S::queries * kAhead < G) {
            load(k, h0 + S::queries * kAhead);
          } else if (w_at + step_w < p.works) {
            k = e4_work<G>(p, w_at + step_w);
            load(k, who);
          }
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const int h = h0 + u * S::queries;
            if (h >= G) continue;
            const uint32_t in[4] = {now[u].x, now[u].y, now[u].z, now[u].w};
            uint32_t most = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) most = max_two(most, in[j] & 0x7fff7fffu);
            most = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));
            const uint32_t top = __float_as_uint(Two<E>::get(most).x);
            // the largest in [2^7, 2^8) units; a query that is not finite is NaN throughout
            const bool bad = top >= 0x7f800000u;
            const int exponent = max(static_cast<int>(top >> 23) - 127 - 7, -120);
            const float over = __uint_as_float(static_cast<uint32_t>(127 - exponent) << 23);
            if (lane == 0) sh.unit[nw & 3][h] = h < heads ? __uint_as_float(static_cast<uint32_t>(127 + exponent) << 23) : 0.0f;
            uint32_t x[4];  // in fp16: exact from 2^-14 units on, below the last term's steps
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 y = Two<E>::get(in[j]);
              x[j] = half_two(y.x * over, y.y * over);
            }
            if (bad) {
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = 0x7fff7fffu;
            }
            if (lane * 8 >= p.d_blocks * 128) continue;
#pragma unroll
            for (int t = 0; t < TERMS; ++t) {
              uint32_t two[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                two[j] = e4m3_of_half2(x[j]);
                if (t + 1 < TERMS) x[j] = rest16(x[j], half2_of_e4m3(two[j]));
              }
              *reinterpret_cast<uint2*>(to + (lane >> 4) * q_block + swizzled(t * G + h, (lane >> 1) & 7) + (lane & 1) * 8) =
                  make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full[qb]), mbar_arrive(&sh.units[nw & 3]);
      }
    }
    __syncwarp();
    registers<S::query_regs, S::regs>();
  } else {
    registers<S::regs, S::softmax_regs>();
    // ---- softmax: thread `e` of a set has entry e of each tile, for the set's heads ----
    const int set = warp >> 2, e = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t p_mine = p_at + e * 16 + (HS == 16 ? set * (kEntries * 16) : 0);
    float* nref = sh.nref + set * HS;
    const uint64_t* held = reinterpret_cast<const uint64_t*>(nref);
    int n = 0, nw = 0, note = 0;
    for (uint32_t w_at = first_w; w_at < p.works; w_at += step_w, ++nw, n += tiles) {
      const E4Work k = e4_work<G>(p, w_at);
      const int heads = min(max(k.heads - set * HS, 0), HS);
      const uint64_t* unit = reinterpret_cast<const uint64_t*>(sh.unit[nw & 3] + set * HS);
      const float* slopes = a.slopes != nullptr ? a.slopes + k.head0 + set * HS : nullptr;
      uint64_t sum[HS / 2];  // of the weights of two heads
#pragma unroll
      for (int h = 0; h < HS / 2; ++h) sum[h] = 0;
      if (e < HS) nref[e] = e < heads ? 0.0f : -kNoHead;
      bool ok = true, fresh = true;  // a head of the set has seen nothing yet
      if (tiles > 0) ok = wait_or_stop(&sh.units[nw & 3], (nw >> 2) & 1, stop);
      set_sync(set);
      // A wait that ran out ends nothing here: the set's threads stay together, and
      // what they compute from then on becomes NaN.
      for (int i = 0; i < tiles; ++i) {
        const int at = n + i;
        const Notes& notes = *reinterpret_cast<const Notes*>(smem + p.note_at + note * p.note_bytes);
        ok = wait_or_stop(&sh.s_full[at & 7], (at >> 3) & 1, stop) && ok;
        tc_fence_after();
        const float ks = notes.ks[e], vs = notes.vs[e];
        const bool seen = (notes.seen[e >> 5] >> (e & 31)) & 1;
        const float log_vs = log2_fast(fmaxf(fabsf(vs), kLeast));
        // Logits in units of log 2, two heads at a time, less the references; once more where
        // those moved so far that what is left after them was rounded away.
        uint64_t z[HS / 2];
        bool moved = false;  // sums have to follow
#pragma unroll 1
        for (bool more = true, again = true; more;) {
          {
            uint32_t v[TERMS][HS];
            const uint32_t s_at = tmem_s + (at & 1) * N + lanes + set * HS;
#pragma unroll
            for (int t = 0; t < TERMS; ++t) tmem_ld(v[t], s_at + t * G);
#pragma unroll
            for (int t = 0; t < TERMS; ++t) tmem_wait_ld(v[t]);
            auto of = [&](int t, int h) { return pair(__uint_as_float(v[t][2 * h]), __uint_as_float(v[t][2 * h + 1])); };
#pragma unroll
            for (int h = 0; h < HS / 2; ++h) {
              z[h] = of(TERMS - 1, h);
#pragma unroll
              for (int t = TERMS - 2; t >= 0; --t) z[h] = fma2(z[h], twice(0x1p-4f), of(t, h));
            }
          }
          if (a.softcap > 0.0f) {
            // the second form only where a logit of the warp needs it
            float most = 0.0f;
#pragma unroll
            for (int h = 0; h < HS / 2; ++h) {
              z[h] = mul2(z[h], mul2(twice(ks), unit[h]));
              const float2 y = both(z[h]);
              most = fmaxf(most, fmaxf(fabsf(y.x), fabsf(y.y)));
            }
            const bool bent = __any_sync(0xffffffffu, !(most * fabsf(p.scale_over_cap) < kBent));
#pragma unroll
            for (int h = 0; h < HS / 2; ++h) {
              const uint64_t u = mul2(z[h], twice(p.scale_over_cap));
              float2 y = capped_low(z[h], u, p.scale_log2e);
              if (bent) {
                const float2 in = both(u), high = capped_high(u, p.cap_log2e);
                if (!(fabsf(in.x) < kBent)) y.x = high.x;
                if (!(fabsf(in.y) < kBent)) y.y = high.y;
              }
              z[h] = pair(y.x, y.y);
            }
          }
          if (slopes != nullptr) {
            const float away = notes.away[e] * kLog2e;
            const uint64_t factor = twice(ks * p.scale_log2e);
#pragma unroll
            for (int h = 0; h < HS / 2; ++h) {
              if (!(a.softcap > 0.0f)) z[h] = mul2(z[h], mul2(factor, unit[h]));
              const uint64_t s = pair(2 * h < heads ? slopes[2 * h] : 0.0f, 2 * h + 1 < heads ? slopes[2 * h + 1] : 0.0f);
              z[h] = fma2(s, twice(away), z[h]);
            }
          }
          // less the references; times the scales where neither cap nor slopes took them
          const bool plain = !(a.softcap > 0.0f) && slopes == nullptr;
          const uint64_t factor = twice(ks * p.scale_log2e);
          if (plain) {
#pragma unroll
            for (int h = 0; h < HS / 2; h += 2) {
              const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(&unit[h]), r = *reinterpret_cast<const ulonglong2*>(&held[h]);
              z[h] = fma2(z[h], mul2(factor, u.x), r.x), z[h + 1] = fma2(z[h + 1], mul2(factor, u.y), r.y);
            }
          } else {
#pragma unroll
            for (int h = 0; h < HS / 2; h += 2) {
              const ulonglong2 r = *reinterpret_cast<const ulonglong2*>(&held[h]);
              z[h] = add2(z[h], r.x), z[h + 1] = add2(z[h + 1], r.y);
            }
          }
          float high = -FLT_MAX;
#pragma unroll
          for (int h = 0; h < HS / 2; ++h) {
            const float2 y = both(z[h]);
            high = fmaxf(high, fmaxf(y.x, y.y));
          }
          if (!fresh && !set_any(set, seen && high + log_vs > kLogLimit)) break;
          // Move the references, by whole numbers.
          const float low = __int_as_float(0xff800000);
          float w[HS];  // a NaN is no maximum
#pragma unroll
          for (int h = 0; h < HS; ++h) {
            const float2 y = both(z[h / 2]);
            w[h] = seen ? fmaxf((h & 1 ? y.y : y.x) + log_vs, low) : low;
          }
          const float top = max_lanes<HS>(w, lane);
          if (lane % (32 / HS) == 0) sh.most[warp][lane / (32 / HS)] = top;
          set_sync(set);
          bool far = false;
          if (e < HS) {
            const float(*m)[HS] = &sh.most[set * 4];
            const float top = fmaxf(fmaxf(m[0][e], m[1][e]), fmaxf(m[2][e], m[3][e]));
            // An infinite logit makes a reference of NaN, which all that follows takes on.
            const float by = top > FLT_MAX ? __int_as_float(0x7fc00000) : ceilf(top) - kTop;
            // From nothing to where the first logits are; then up where a weight is too large:
            // what a head's references are depends on its own logits alone.
            const bool first = begins(nref[e]), moves = e < heads && (first ? top > low : top > kLogLimit);
            sh.step[set * HS + e] = moves ? -by : 0.0f;
            const float factor = moves && !first ? exp2_fast(-by) : 1.0f;
            sh.factor[set * HS + e] = again ? factor : factor * sh.factor[set * HS + e];
            if (moves) nref[e] = nref[e] == by ? -0.0f : nref[e] - by;
            far = moves && !first && by > kFar;
          }
          more = i > 0 && again && set_any(set, far);
          again = false;
          fresh = set_any(set, e < heads && begins(nref[e]));
          const uint64_t* step = reinterpret_cast<const uint64_t*>(sh.step + set * HS);
#pragma unroll
          for (int h = 0; h < HS / 2; ++h) z[h] = add2(z[h], step[h]);
          moved = i > 0;
        }
        if (moved) {  // the sums follow; O^T's columns do below, when the weights are out
          const ulonglong2* factor = reinterpret_cast<const ulonglong2*>(sh.factor + set * HS);
#pragma unroll
          for (int h = 0; h < HS / 4; ++h) {
            const ulonglong2 f = factor[h];
            sum[2 * h] = mul2(sum[2 * h], f.x), sum[2 * h + 1] = mul2(sum[2 * h + 1], f.y);
          }
        }
        if (notes.seen[e >> 5] != 0xffffffffu && !seen) {
#pragma unroll
          for (int h = 0; h < HS / 2; ++h) z[h] = twice(__int_as_float(0xff800000));
        }
        uint32_t words[TERMS][HS / 4];  // the weights' terms, four heads each
#pragma unroll
        for (int h = 0; h < HS / 2; ++h) {
          const float2 y = both(z[h]);
          const uint64_t w = pair(exp2_fast(y.x), exp2_fast(y.y));
          sum[h] = add2(sum[h], w);
          const float2 scaled = both(mul2(w, twice(vs)));
          uint32_t x = half_two(scaled.x, scaled.y);
#pragma unroll
          for (int t = 0; t < TERMS; ++t) {
            const uint32_t two = e4m3_of_half2(x);
            if (t + 1 < TERMS) x = rest16(x, half2_of_e4m3(two));
            words[t][h / 2] = h & 1 ? words[t][h / 2] | two << 16 : two;
          }
        }
        const uint32_t to = p_mine + (at & 1) * S::p_bytes;
        if constexpr (HS == 16) {
#pragma unroll
          for (int t = 0; t < TERMS; ++t)
            put16(to + t * SETS * (kEntries * 16), words[t][0], words[t][1], words[t][2], words[t][3]);
        } else {  // two terms of eight heads a unit; the other half of the third's is nobody's
          put16(to, words[0][0], words[0][1], words[1][0], words[1][1]);
          if constexpr (TERMS == 3) put16(to + kEntries * 16, words[2][0], words[2][1], 0, 0);
        }
        if (moved) {
          ok = wait_or_stop(&sh.pv_done[(at - 1) & 7], ((at - 1) >> 3) & 1, stop) && ok;
          tc_fence_after();
          uint32_t which = __ballot_sync(0xffffffffu, lane < HS && sh.factor[set * HS + (lane & (HS - 1))] != 1.0f);
          // one head's columns at a time: few move, and there are no registers for more
#pragma unroll 1
          for (; which != 0; which &= which - 1) {
            const int h = set * HS + __ffs(which) - 1;
            const float f = sh.factor[h];
            uint32_t v[2][TERMS];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int t = 0; t < TERMS; ++t)
                if (m < p.v_blocks) tmem_ld(v[m][t], tmem_o + m * N + lanes + t * G + h);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int t = 0; t < TERMS; ++t) tmem_wait_ld(v[m][t]);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int t = 0; t < TERMS; ++t)
                if (m < p.v_blocks) tmem_st(tmem_o + m * N + lanes + t * G + h, __float_as_uint(__uint_as_float(v[m][t]) * f));
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[at & 7]);
        if (++note == p.notes) note = 0;
      }

      // ---- end of a work ----
      // A barrier that was given up may look over to who comes to it eight tiles on, in
      // a later work: those are lost whole.
      if (*stop != 0) ok = false;
      float sums[HS];
#pragma unroll
      for (int h = 0; h < HS; ++h) {
        const float2 y = both(sum[h / 2]);
        sums[h] = ok ? h & 1 ? y.y : y.x : __int_as_float(0x7fc00000);
      }
      const float part = sum_lanes<HS>(sums, lane);
      if (lane % (32 / HS) == 0) sh.sum[warp][lane / (32 / HS)] = part;
      set_sync(set);
      float total = 0.0f;
      if (e < HS) {
        const float(*m)[HS] = &sh.sum[set * 4];
        total = (m[0][e] + m[1][e]) + (m[2][e] + m[3][e]);
        if (cluster > 1)
          sh.head_ref[set * HS + e] = begins(nref[e]) ? __int_as_float(0xff800000) : -nref[e], sh.head_sum[set * HS + e] = total;
        else
          sh.inverse[set * HS + e] = e4_inverse(total);
      }
      set_sync(set);
      if (cluster == 1 && a.lse != nullptr && e < heads) a.lse[k.row * a.Hq + k.head0 + set * HS + e] = e4_logsum(-nref[e], total);
      if (tiles > 0 && !wait_or_stop(&sh.pv_done[(n + tiles - 1) & 7], ((n + tiles - 1) >> 3) & 1, stop)) ok = false;
      tc_fence_after();
      // A thread has one element of every head: two bytes a store, side by side in a warp.
      const int pad = p.v_blocks * 128;
      float* rows = reinterpret_cast<float*>(smem) + set * HS * pad;
      for (int m = 0; m < p.v_blocks; ++m) {
        uint64_t x[HS / 2];  // of two heads
#pragma unroll
        for (int h = 0; h < HS / 2; ++h) x[h] = 0;
        if (tiles > 0) {
          uint32_t v[TERMS][HS];
          const uint32_t o_at = tmem_o + m * N + lanes + set * HS;
#pragma unroll
          for (int t = 0; t < TERMS; ++t) tmem_ld(v[t], o_at + t * G);
#pragma unroll
          for (int t = 0; t < TERMS; ++t) tmem_wait_ld(v[t]);
          auto of = [&](int t, int h) { return pair(__uint_as_float(v[t][2 * h]), __uint_as_float(v[t][2 * h + 1])); };
#pragma unroll
          for (int h = 0; h < HS / 2; ++h) {
            x[h] = of(TERMS - 1, h);
#pragma unroll
            for (int t = TERMS - 2; t >= 0; --t) x[h] = fma2(x[h], twice(0x1p-4f), of(t, h));
          }
        }
        if (!ok) {
#pragma unroll
          for (int h = 0; h < HS / 2; ++h) x[h] = twice(__int_as_float(0x7fc00000));
        }
        const int d = m * 128 + e;
        if (cluster > 1) {
#pragma unroll
          for (int h = 0; h < HS / 2; ++h) {
            const float2 y = both(x[h]);
            rows[2 * h * pad + d] = y.x, rows[(2 * h + 1) * pad + d] = y.y;
          }
        } else if (d < a.Dv) {
#pragma unroll
          for (int h = 0; h < HS; h += 4) {
            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&sh.inverse[set * HS + h]);
            const float2 y = both(mul2(x[h / 2], f.x)), z = both(mul2(x[h / 2 + 1], f.y));
            E* row = static_cast<E*>(a.out) + (k.row * a.Hq + k.head0 + set * HS + h) * a.Dv + d;
            if (h < heads) row[0] = E(y.x);
            if (h + 1 < heads) row[a.Dv] = E(y.y);
            if (h + 2 < heads) row[2 * a.Dv] = E(z.x);
            if (h + 3 < heads) row[3 * a.Dv] = E(z.y);
          }
        }
      }
      tc_fence_before();  // O is read: the next work's first weights say so
      set_sync(set);      // and what the set shares
    }
    registers<S::softmax_regs, S::regs>();
  }

  __syncthreads();
  if (*stop != 0) {  // a wait ran out: nobody may have waited for what is in flight
    if (one) mma_drain(&sh.drained);
    copy_commit();
    copy_wait<0>();
    __syncthreads();
  }
  if (cluster > 1) {
    // ---- join the CTAs: four outputs a thread, all reads of all CTAs in flight together ----
    const E4Work k = e4_work<G>(p, first_w);
    const int pad = p.v_blocks * 128;
    E* out = static_cast<E*>(a.out) + (k.row * a.Hq + k.head0) * a.Dv;
    cluster_sync();
    const uint32_t ref_addr = smem_addr(sh.head_ref), sum_addr = smem_addr(sh.head_sum);
    const int fours = a.Dv / 4, outputs = k.heads * fours;
    for (int i = static_cast<int>(rank) * S::threads + threadIdx.x; i < outputs; i += cluster * S::threads) {
      const int h = i / fours, c = (i - h * fours) * 4;
      float m[8], l[8], all = __int_as_float(0xff800000), total = 0.0f;
      float4 u[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const uint32_t from = r < cluster ? r : 0;
        m[r] = __uint_as_float(ld_dsmem_u32(map_rank(ref_addr + 4 * h, from)));
        l[r] = __uint_as_float(ld_dsmem_u32(map_rank(sum_addr + 4 * h, from)));
        u[r] = ld_dsmem_f4(map_rank(base + 4 * (h * pad + c), from));
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) all = fmaxf(all, m[r]);
      float4 x = {};
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (r >= cluster) continue;
        const float f = m[r] == all ? 1.0f : exp2_fast(m[r] - all);
        total += l[r] * f;
        x.x += u[r].x * f, x.y += u[r].y * f, x.z += u[r].z * f, x.w += u[r].w * f;
      }
      const float f = e4_inverse(total);
      *reinterpret_cast<uint2*>(out + static_cast<int64_t>(h) * a.Dv + c) =
          make_uint2(Pack<E>::two(x.x * f, x.y * f), Pack<E>::two(x.z * f, x.w * f));
      if (c == 0 && a.lse != nullptr) a.lse[k.row * a.Hq + k.head0 + h] = e4_logsum(all, total);
    }
    cluster_sync();  // the others may still read this CTA's rows
  }
  if (warp == S::mma) {
    tc_fence_after();
    tmem_free(sh.tmem, p.tmem_cols);
  }
}

template <typename E, int G>
topk_status launch_heads(const sparse_attention_e4m3_args& args, int dev, int sm_count, cudaStream_t stream) {
  using S = Shape<E, G>;
  const sparse_attention_args& a = args.attention;
  E4Params p = {};
  p.a = a;
  p.k_scales = args.k_scales, p.v_scales = args.v_scales;
  p.blocks = args.blocks, p.block = args.blocks > 0 ? a.page_size / args.blocks : 1;
  p.heads = a.Hq / a.Hkv;
  p.h_tiles = (p.heads + G - 1) / G;
  p.scale_log2e = finite(static_cast<double>(a.scale) * kLog2e);
  if (a.softcap > 0.0f) {
    p.scale_over_cap = finite(static_cast<double>(a.scale) / a.softcap);
    p.cap_log2e = finite(static_cast<double>(a.softcap) * kLog2e);
  }
  p.page_shift = p.block_shift = -1;
  for (int i = 0; i < 31; ++i) {
    if (a.page_size == 1 << i) p.page_shift = i;
    if (p.block == 1 << i) p.block_shift = i;
  }
  p.pages = a.num_pages < INT32_MAX ? static_cast<uint32_t>(a.num_pages) : INT32_MAX;
  p.table_width = a.table_width < INT32_MAX ? static_cast<uint32_t>(a.table_width) : INT32_MAX;
  p.d_blocks = (a.D + 127) / 128, p.v_blocks = (a.Dv + 127) / 128, p.d_steps = (a.D + 31) / 32;
  p.shared = a.k == a.v && a.Dv <= a.D && a.k_page_stride == a.v_page_stride && a.k_token_stride == a.v_token_stride &&
             a.k_head_stride == a.v_head_stride;
  p.q_vector = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && a.q_seq_stride % 8 == 0 && a.q_token_stride % 8 == 0 &&
               a.q_head_stride % 8 == 0;
  p.k_bytes = kEntries * 128 * p.d_blocks;
  p.v_bytes = p.shared ? 0 : kEntries * 128 * p.v_blocks;
  p.note_bytes = static_cast<int32_t>(a.slopes != nullptr ? sizeof(Notes) : offsetof(Notes, away));
  const int columns = (kBufs + p.v_blocks) * S::N;
  p.tmem_cols = 32;
  while (p.tmem_cols < columns) p.tmem_cols *= 2;
  using Shared = E4Shared<G, S::sets, S::set_heads>;
  const int q_bytes = kBufs * S::rows * 128 * p.d_blocks, p_bytes = kBufs * S::p_bytes;
  const int fixed = q_bytes + p_bytes + static_cast<int>(sizeof(Shared)) + kBufs * p.note_bytes;
  const int stage = p.k_bytes + p.v_bytes + p.note_bytes;
  const int join = G * p.v_blocks * 128 * 4;  // rows for the other CTAs, over the queries and the rings
  // Two CTAs share an SM where two stages each fit, else one has as many stages as fit.
  const int half = kMaxShared / 2 - 1024;
  const bool two = S::per_sm == 2 && fixed + 2 * stage <= half && p.tmem_cols <= 256 && join <= half - fixed + q_bytes;
  const int room = (two ? half : kMaxShared) - fixed;
  p.k_stages = room / stage < kMaxStages ? room / stage : kMaxStages;
  if (p.k_stages < (p.shared ? 2 : 1)) return TOPK_EINVAL;  // S of a tile goes ahead of O^T of the one before
  p.v_stages = p.shared ? 0 : p.k_stages;
  if (!p.shared && p.k_stages < kMaxStages && room - p.k_stages * stage >= p.v_bytes) ++p.v_stages;
  p.notes = p.k_stages + kBufs;
  p.k_at = q_bytes;
  p.v_at = p.k_at + p.k_stages * p.k_bytes;
  int end = p.v_at + p.v_stages * p.v_bytes;
  if (end < join) end = (join + 1023) / 1024 * 1024;
  p.p_at = end;
  p.note_at = p.p_at + p_bytes;
  p.shared_at = p.note_at + (p.notes * p.note_bytes + 15) / 16 * 16;
  // CTAs that share an SM must find their TMEM free (see sparse_attention.cu): with up to
  // 256 columns each takes more than a third of the shared memory, with more all of it.
  size_t bytes = static_cast<size_t>(p.shared_at) + sizeof(Shared);
  if (bytes > kMaxShared) return TOPK_EINVAL;
  const size_t floor_bytes = p.tmem_cols > 256 ? kMaxShared : 77 * 1024;
  if (bytes < floor_bytes) bytes = floor_bytes;
  const int64_t work = static_cast<int64_t>(a.B) * a.T * a.Hkv * p.h_tiles;
  if (work > INT32_MAX) return TOPK_EINVAL;
  p.works = static_cast<uint32_t>(work);
  // Few rows: share each over the CTAs that would idle, down to two tiles each. Long lists: share
  // each, so that a CTA, which has references of its own, has kLongest entries: what its last steps
  // lose is relative to its own largest weight, so all together lose what one list of 2048 does. A
  // CTA then ends with its row: 512 rows of 64 heads over 4096 entries 309 us (243 unshared), 64 x 8
  // heads' lists of 4096 118 (100).
  const int64_t slots = static_cast<int64_t>(sm_count) * (two ? 2 : 1);
  const int tiles = a.K / kEntries + (a.K % kEntries != 0);
  int cluster = 1;
  while (cluster < 8 && ((work * cluster * 2 <= slots && cluster * 4 <= tiles) || tiles > cluster * (kLongest / kEntries)))
    cluster *= 2;
  const int64_t grid = cluster == 1 && work > slots ? slots : work * cluster;
  if (grid > INT32_MAX || (work / grid + 1) * tiles > INT32_MAX) return TOPK_EINVAL;  // a CTA counts its tiles
  constexpr auto kernel = cache_attention_kernel<E, G>;
  // What the groups of warps trade is what the launch brings.
  topk_status st = has_registers<kernel>(S::regs);
  if (st != TOPK_OK) return st;
  st = allow_shared<kernel>(dev);
  if (st != TOPK_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(S::threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  return status_of(cudaLaunchKernelEx(&cfg, kernel, p, cluster));
}

// The least padded heads that hold those of a key head, or tiles of the most: columns cost the
// softmax warps whether they hold a head or not, and a tile more reads the entries once more.
template <typename E>
topk_status launch_cache_attention(const sparse_attention_e4m3_args& a, int dev, int sm_count, cudaStream_t stream) {
  const int heads = a.attention.Hq / a.attention.Hkv;
  if (heads <= 8) return launch_heads<E, 8>(a, dev, sm_count, stream);
  if (heads <= 16) return launch_heads<E, 16>(a, dev, sm_count, stream);
  if constexpr (std::is_same<E, __nv_bfloat16>::value)  // TMEM has no room for three terms of 64 heads
    if (heads > 32) return launch_heads<E, 64>(a, dev, sm_count, stream);
  return launch_heads<E, 32>(a, dev, sm_count, stream);
}

}  // namespace
}  // namespace tki
