// Attention over selected entries of a paged cache in 8 bits
// (include/sparse_cache.h, sparse_attention_e4m3).
//
// The products. Entries go from the cache into the tensor cores as they are, in
// E4M3, with no conversion on the way: kind f8f6f4 takes both operands in 8 bits,
// so queries and weights are split into E4M3 terms, x = u (t0 + t1 / 16 + t2 / 256),
// each the rounded rest of those before. A term adds five bits (four and the
// rest's sign): two hold 9, a bf16 query exactly; three hold 14, an fp16 query
// exactly. Two terms of a weight round it to 2^-9 of itself, half a step of bf16's,
// three are good to fp16's 2^-11, which it is rounded to first. A query's unit u is a
// power of two, its head's own.
//
// The tile. 128 entries are the rows of both products and their (term, head) pairs the
// columns: S = K Q^T, and O^T += V^T P with P read along the entries. So few heads a key
// head cost few columns instead of empty rows, each term has sums of its own, which are
// joined with their factors in FP32 registers, and one thread has one entry: its scales,
// mask and position are scalars, and every exponential is one thread's own.
//
// The scales. A key's scale multiplies its logit. A value's multiplies its weight
// before that is split: w = 2^(z - r) s. The reference r of a head is moved, for all
// threads at once, when a weight would pass E4M3's 448, and then to leave the largest
// in (2^6, 2^7]: a weight's terms keep their digits down to 2^-14 / 2^6 of the largest
// one's (three terms: 2^-18). The sum that divides adds the weights in FP32, unrounded
// and without the values' scales. r is a whole number, so moving it is exact.
//
// The rest is as in sparse_attention.cu: entries gathered by 16-byte copies into rings
// of keys and values, few rows shared by a cluster whose CTAs join through distributed
// shared memory, CTAs that stay for several rows where there are many.
//
// Warps: 4 softmax warps for each 16 heads (8: G = 8), one entry a thread; 8 that gather; one
// thread each for S and for O; two that split the queries of the next row.
#include <cuda_runtime.h>

#include <cfloat>
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
constexpr int kGather = 8, kQuery = 2;  // warps
constexpr int kMaxStages = 6;
constexpr int kBufs = 2;                  // buffers of scores in TMEM
constexpr int kMaxNotes = kMaxStages + kBufs;  // see E4Params::notes
constexpr float kNothing = -1073741824.0f;  // a reference below any logit in use; its negative for heads that are none
constexpr float kLimit = 448.0f;
constexpr float kLeast = 0x1p-60f;  // values' scales below count as this for the reference

template <typename E, int G>
struct Shape {
  static constexpr int terms = std::is_same<E, __nv_bfloat16>::value ? 2 : 3;
  static constexpr int set_heads = G < 16 ? G : 16;  // of one set of four softmax warps
  static constexpr int sets = G / set_heads;
  static constexpr int rows = terms * G;              // (term, head) pairs
  static constexpr int N = (rows + 15) / 16 * 16;     // columns; those past the rows come from whatever follows them
  static constexpr int q_bufs = G <= 16 ? 2 : 1, p_bufs = G <= 16 ? 1 : 2;
  static constexpr int softmax = 4 * sets;            // warps
  static constexpr int mma = softmax + kGather, query = mma + 2;
  static constexpr int threads = (query + kQuery) * 32;
  static constexpr int per_sm = G <= 16 ? 2 : 1;
};

struct E4Params {
  sparse_attention_args a;
  const float* k_scales;
  const float* v_scales;
  int32_t block, blocks;     // entries of a block, blocks a page
  int32_t heads, h_tiles;    // query heads per key head, tiles of G of them
  uint32_t works;            // (row, key head, tile of heads)
  int32_t d_blocks, v_blocks, d_steps;  // 128-byte blocks of an entry, 32-byte steps of its keys
  int32_t shared;            // v is a prefix of k's entries
  int32_t page_shift, block_shift;  // log2, or -1
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
  float ref[G], factor[G], inverse[G];
  float unit[4][G];  // of the queries, of the last four works
  float most[SETS * 4][HS], sum[SETS * 4][HS];
  float head_ref[G], head_sum[G];  // for the other CTAs of a cluster
  uint64_t k_full[kMaxStages], v_full[kMaxStages], noted[kMaxNotes];
  uint64_t q_full[2], q_empty[2], units[4];
  // Of tile i at i % 8: scores there, weights there, products with v done.
  uint64_t s_full[8], p_full[8], pv_done[8];
  uint64_t o_free;
  uint64_t drained[2];
  uint32_t tmem;
  uint32_t stop;
};

struct E4Work {
  int g, heads, head0;
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

// A float as an integer of the same order, and back.
__device__ __forceinline__ int32_t ordered(float x) {
  const int32_t i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_ordered(int32_t i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

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
// 16 (x - y), exactly where x - y is what a term of x leaves.
__device__ __forceinline__ uint32_t rest16(uint32_t x, uint32_t y) {
  const __half2 a = *reinterpret_cast<const __half2*>(&x), b = *reinterpret_cast<const __half2*>(&y);
  const __half2 r = __hmul2(__hsub2(a, b), __float2half2_rn(16.0f));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void put_byte(uint32_t at, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// 1 / a sum of weights, zero where nothing is seen; and its logarithm with the reference.
__device__ __forceinline__ float e4_inverse(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }
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

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.k_stages; ++i) mbar_init(&sh.k_full[i], p.shared ? 256 : 128);
    for (int i = 0; i < p.v_stages; ++i) mbar_init(&sh.v_full[i], 128);
    for (int i = 0; i < p.notes; ++i) mbar_init(&sh.noted[i], 128 + 4);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.q_full[i], kQuery * 32), mbar_init(&sh.q_empty[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&sh.units[i], kQuery * 32);
    for (int i = 0; i < 8; ++i)
      mbar_init(&sh.s_full[i], 1), mbar_init(&sh.p_full[i], 128 * SETS), mbar_init(&sh.pv_done[i], 1);
    mbar_init(&sh.o_free, 128 * SETS);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.drained[i], 1);
    sh.stop = 0;
    fence_mbar_init();
  }
  if (warp == S::mma) tmem_alloc(&sh.tmem, p.tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_s = sh.tmem, tmem_o = tmem_s + kBufs * N;
  volatile uint32_t* stop = &sh.stop;
  bool one = false;  // a thread that issues products

  if (warp >= S::softmax && warp < S::mma) {
    // ---- gather ----
    // Four warps fetch the tile's keys, 32 entries each, and note what belongs to
    // them; four their values, or the second half of their blocks when shared.
    const int w = warp - S::softmax, part = w & 3;
    const bool second = w >= 4, values = second && !p.shared;
    const int split = (p.d_blocks + 1) / 2;
    const int c0 = second && p.shared ? split : 0;
    const int c1 = values ? p.v_blocks : !second && p.shared ? split : p.d_blocks;
    // 16-byte units of an entry: those that it has, and those that are read (a whole
    // step of the keys' product, of the values those that it has)
    const int units = (values ? a.Dv : a.D) / 16, read = values ? units : p.d_steps * 2;
    const int64_t head_stride = values ? a.v_head_stride : a.k_head_stride;
    const int64_t page_stride = values ? a.v_page_stride : a.k_page_stride;
    const int64_t token_stride = values ? a.v_token_stride : a.k_token_stride;
    uint64_t* full = values ? sh.v_full : sh.k_full;
    uint64_t* used = values || p.shared ? sh.pv_done : sh.s_full;  // when a tile's stage is free
    const int stages = values ? p.v_stages : p.k_stages, stage_bytes = values ? p.v_bytes : p.k_bytes;
    const uint32_t unit16 = lane & 7, sub = lane >> 3;
    const uint32_t at = (values ? v_ring : k_ring) + (part * 32 + sub) * 128;
    const uint32_t even = (unit16 ^ sub) << 4, odd = (unit16 ^ (sub + 4)) << 4;
    const bool some = a.page_size > 0 && a.num_pages > 0;
    bool ok = true;
    int stage = 0, note = 0, n = 0;
    for (uint32_t w_at = first_w; w_at < p.works && ok; w_at += step_w, n += tiles) {
      const E4Work k = e4_work<G>(p, w_at);
      const int32_t* indices = a.indices + k.row * a.K;
      const int32_t* table = a.page_table != nullptr ? a.page_table + k.b * a.table_stride : nullptr;
      const int32_t last = a.query_positions != nullptr ? a.query_positions[k.row] : INT32_MAX;
      const int32_t first = a.first != nullptr ? max(a.first[k.row], 0) : 0;
      // Each lane looks up one entry of a tile, its index two tiles ahead, its page id one.
      auto index_of = [&](int i) -> int32_t {
        const int64_t j = (static_cast<int64_t>(i) * cluster + rank) * kEntries + part * 32 + lane;
        return i < tiles && j < a.K && some ? indices[j] : -1;
      };
      auto page_index = [&](int32_t pos) -> uint32_t {
        return p.page_shift >= 0 ? static_cast<uint32_t>(pos) >> p.page_shift
                                 : static_cast<uint32_t>(pos) / static_cast<uint32_t>(a.page_size);
      };
      auto page_of = [&](int32_t pos) -> uint32_t {  // ~0: not seen
        if (pos < first || pos > last) return 0xffffffffu;
        const uint32_t page = page_index(pos);
        return table == nullptr ? page : page < p.table_width ? static_cast<uint32_t>(table[page]) : 0xffffffffu;
      };
      int32_t pos = index_of(0), pos1 = index_of(1);
      uint32_t page = page_of(pos);
      // an empty cache has no address: nothing is read from the one it gets
      const char* nowhere = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(a.q) & ~static_cast<uintptr_t>(15));
      const char* mine = some ? static_cast<const char*>(values ? a.v : a.k) + k.g * head_stride + unit16 * 16 : nowhere;
      for (int i = 0; i < tiles; ++i) {
        const int32_t pos2 = index_of(i + 2);
        const uint32_t page1 = page_of(pos1);
        const bool seen = page < p.pages;
        const uint32_t place = static_cast<uint32_t>(pos) - page_index(pos) * static_cast<uint32_t>(a.page_size);
        const int64_t entry = seen ? page * page_stride + place * token_stride : 0;
        const uint32_t bits = __ballot_sync(0xffffffffu, seen);
        const int before = n + i - stages;
        ok = before < 0 || wait_or_stop(&used[before & 7], (before >> 3) & 1, stop);
        if (!ok) break;
        const uint32_t dst = at + stage * stage_bytes;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const char* from = mine + __shfl_sync(0xffffffffu, entry, 4 * j + sub);
          const bool there = (bits >> (4 * j + sub)) & 1;  // what is not seen is zeros
          for (int c = c0; c < c1; ++c) {
            const int u = c * 8 + static_cast<int>(unit16);
            if (u < read)
              copy_bytes(dst + c * (kEntries * 128) + j * 512 + (j & 1 ? odd : even), u < units ? from + c * 128 : mine,
                         there && u < units ? 16 : 0);
          }
        }
        copy_arrive(&full[stage]);
        if (!second) {
          Notes& notes = *reinterpret_cast<Notes*>(smem + p.note_at + note * p.note_bytes);
          const int e = part * 32 + lane;
          const uint32_t block = p.block_shift >= 0 ? place >> p.block_shift : place / static_cast<uint32_t>(p.block);
          const int64_t unit = seen ? (static_cast<int64_t>(page) * p.blocks + block) * a.Hkv + k.g : 0;
          copy4(smem_addr(&notes.ks[e]), some ? reinterpret_cast<const char*>(p.k_scales + unit) : nowhere, seen);
          copy4(smem_addr(&notes.vs[e]), some ? reinterpret_cast<const char*>(p.v_scales + unit) : nowhere, seen);
          copy_arrive(&sh.noted[note]);
          if (a.slopes != nullptr) notes.away[e] = static_cast<float>(seen ? pos - last : 0);
          if (lane == 0) notes.seen[part] = bits;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.noted[note]);
        }
        pos = pos1, pos1 = pos2, page = page1;
        if (++stage == stages) stage = 0;
        if (++note == p.notes) note = 0;
      }
    }
    copy_commit();
    copy_wait<0>();
  } else if (warp == S::mma) {
    // ---- S = K Q^T, by one thread ----
    one = elect_one();
    if (tiles > 0 && one) {
      const uint32_t desc = mma_desc(0, N);
      const uint64_t q_desc = operand_desc(base), k_desc = operand_desc(k_ring);
      int stage = 0, turn_of = 0, n = 0, nw = 0;
      bool ok = true;
      for (uint32_t w_at = first_w; w_at < p.works && ok; w_at += step_w, ++nw) {
        const int qb = nw % S::q_bufs;
        const uint64_t qd = q_desc + static_cast<uint32_t>(qb * q_bytes >> 4);
        ok = wait_or_stop_one(&sh.q_full[qb], (nw / S::q_bufs) & 1, stop);
        for (int i = 0; i < tiles && ok; ++i, ++n) {
          const int before = n - kBufs;  // whose scores were there
          ok = (before < 0 || wait_or_stop_one(&sh.p_full[before & 7], (before >> 3) & 1, stop)) &&
               wait_or_stop_one(&sh.k_full[stage], turn_of, stop);
          if (!ok) break;
          fence_proxy_async_smem();
          tc_fence_after();
          const uint64_t kd = k_desc + static_cast<uint32_t>(stage * p.k_bytes >> 4);
          const uint32_t to = tmem_s + (n & 1) * N;
          for (int j = 0; j < p.d_steps; ++j) {
            const uint32_t c = j >> 2, in = (j & 3) * 2;
            mma_f8(to, kd + (c * (kEntries * 128 >> 4) + in), qd + (c * (S::rows * 128 >> 4) + in), desc, j > 0);
          }
          mma_commit(&sh.s_full[n & 7]);
          if (++stage == p.k_stages) stage = 0, turn_of ^= 1;
        }
        if (ok) mma_commit(&sh.q_empty[qb]);
      }
    }
    __syncwarp();
  } else if (warp == S::mma + 1) {
    // ---- O^T += V^T P, by another ----
    one = elect_one();
    if (tiles > 0 && one) {
      const uint32_t desc = mma_desc(0, N, false, true);
      const uint64_t v_desc = operand_desc(p.shared ? k_ring : v_ring), p_desc = operand_desc(p_at);
      const int stages = p.shared ? p.k_stages : p.v_stages, stage_bytes = p.shared ? p.k_bytes : p.v_bytes;
      uint64_t* full = p.shared ? sh.k_full : sh.v_full;
      int stage = 0, turn_of = 0, n = 0, nw = 0;
      bool ok = true;
      for (uint32_t w_at = first_w; w_at < p.works && ok; w_at += step_w, ++nw) {
        if (nw > 0) ok = wait_or_stop_one(&sh.o_free, (nw - 1) & 1, stop);
        for (int i = 0; i < tiles && ok; ++i, ++n) {
          ok = wait_or_stop_one(&full[stage], turn_of, stop);
          fence_proxy_async_smem();
          ok = ok && wait_or_stop_one(&sh.p_full[n & 7], (n >> 3) & 1, stop);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = v_desc + static_cast<uint32_t>(stage * stage_bytes >> 4);
          const uint64_t pd = p_desc + static_cast<uint32_t>((n % S::p_bufs) * (S::rows * 128) >> 4);
          for (int m = 0; m < p.v_blocks; ++m)
#pragma unroll
            for (int j = 0; j < kEntries / 32; ++j)
              mma_f8(tmem_o + m * N, vd + static_cast<uint32_t>((m * (kEntries * 128) + j * (32 * 128)) >> 4),
                     pd + static_cast<uint32_t>(j * 2), desc, i + j > 0);
          mma_commit(&sh.pv_done[n & 7]);
          if (++stage == stages) stage = 0, turn_of ^= 1;
        }
      }
    }
    __syncwarp();
  } else if (warp >= S::query) {
    // ---- queries: a power of two for each head and terms in units of it ----
    const int who = warp - S::query;
    int nw = 0;
    bool ok = true;
    for (uint32_t w_at = first_w; tiles > 0 && w_at < p.works; w_at += step_w, ++nw) {
      const E4Work k = e4_work<G>(p, w_at);
      const int qb = nw % S::q_bufs;
      if (nw >= S::q_bufs) ok = wait_or_stop(&sh.q_empty[qb], (nw / S::q_bufs - 1) & 1, stop);
      if (!ok) break;
      unsigned char* to = smem + qb * q_bytes;
      const E* q = static_cast<const E*>(a.q) + k.b * a.q_seq_stride + k.t * a.q_token_stride + k.head0 * a.q_head_stride;
      constexpr int kAhead = 4;
      for (int h0 = who; h0 < G; h0 += kQuery * kAhead) {
        alignas(16) E e[kAhead][8];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int h = h0 + u * kQuery;
          const E* from = q + h * a.q_head_stride + lane * 8;
          const bool real = h < k.heads && lane * 8 < a.D;  // D is a multiple of 16
          if (real && p.q_vector) {
            *reinterpret_cast<uint4*>(e[u]) = *reinterpret_cast<const uint4*>(from);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) e[u][j] = real ? from[j] : E(0.0f);
          }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int h = h0 + u * kQuery;
          if (h >= G) continue;
          float x[8];
          uint32_t most = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] = static_cast<float>(e[u][j]);
            most = max(most, __float_as_uint(x[j]) & 0x7fffffffu);
          }
          most = __reduce_max_sync(0xffffffffu, most);
          // the largest in [2^7, 2^8) units; a query that is not finite is NaN throughout
          const bool bad = most >= 0x7f800000u;
          const int exponent = max(static_cast<int>(most >> 23) - 127 - 7, -120);
          const float over = __uint_as_float(static_cast<uint32_t>(127 - exponent) << 23);
          if (lane == 0) sh.unit[nw & 3][h] = h < k.heads ? __uint_as_float(static_cast<uint32_t>(127 + exponent) << 23) : 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = bad ? __int_as_float(0x7fc00000) : x[j] * over;
          if (lane * 8 < p.d_blocks * 128) {
#pragma unroll
            for (int t = 0; t < TERMS; ++t) {
              uint32_t two[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                two[j] = e4m3_two(x[2 * j], x[2 * j + 1]);
                const float2 y = e4m3_both(two[j]);
                x[2 * j] = (x[2 * j] - y.x) * 16.0f, x[2 * j + 1] = (x[2 * j + 1] - y.y) * 16.0f;
              }
              const int row = t * G + h;
              *reinterpret_cast<uint2*>(to + (lane >> 4) * q_block + swizzled(row, (lane >> 1) & 7) + (lane & 1) * 8) =
                  make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
            }
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&sh.q_full[qb]);
      mbar_arrive(&sh.units[nw & 3]);
    }
  } else {
    // ---- softmax: thread `e` of a set has entry e of each tile, for the set's heads ----
    const int set = warp >> 2, e = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t p_mine = p_at + e;  // of row 0, whose 16-byte units stand in order
    float* ref = sh.ref + set * HS;
    int n = 0, nw = 0, note = 0;
    for (uint32_t w_at = first_w; w_at < p.works; w_at += step_w, ++nw, n += tiles) {
      const E4Work k = e4_work<G>(p, w_at);
      const int heads = min(max(k.heads - set * HS, 0), HS);
      const float* unit = sh.unit[nw & 3] + set * HS;
      const float* slopes = a.slopes != nullptr ? a.slopes + k.head0 + set * HS : nullptr;
      float sum[HS];
#pragma unroll
      for (int h = 0; h < HS; ++h) sum[h] = 0.0f;
      if (e < HS) ref[e] = e < heads ? kNothing : -kNothing;
      bool ok = true;
      if (tiles > 0) ok = wait_or_stop(&sh.units[nw & 3], (nw >> 2) & 1, stop);
      set_sync(set);
      // A wait that ran out ends nothing here: the set's threads stay together, and
      // what they compute from then on becomes NaN.
      for (int i = 0; i < tiles; ++i) {
        const int at = n + i;
        const Notes& notes = *reinterpret_cast<const Notes*>(smem + p.note_at + note * p.note_bytes);
        ok = wait_or_stop(&sh.noted[note], (at / p.notes) & 1, stop) && ok;
        const float ks = notes.ks[e], vs = notes.vs[e];
        const bool seen = (notes.seen[e >> 5] >> (e & 31)) & 1;
        const float away = a.slopes != nullptr ? notes.away[e] : 0.0f;
        ok = wait_or_stop(&sh.s_full[at & 7], (at >> 3) & 1, stop) && ok;
        tc_fence_after();
        float z[HS];
        {
          uint32_t v[TERMS][HS];
          const uint32_t s_at = tmem_s + (at & 1) * N + lanes + set * HS;
#pragma unroll
          for (int t = 0; t < TERMS; ++t) tmem_ld(v[t], s_at + t * G);
#pragma unroll
          for (int t = 0; t < TERMS; ++t) tmem_wait_ld(v[t]);
#pragma unroll
          for (int h = 0; h < HS; ++h) {
            float x = __uint_as_float(v[TERMS - 1][h]);
#pragma unroll
            for (int t = TERMS - 2; t >= 0; --t) x = fmaf(x, 0x1p-4f, __uint_as_float(v[t][h]));
            z[h] = x;
          }
        }
        if (a.softcap > 0.0f) {
#pragma unroll
          for (int h = 0; h < HS; h += 2) {
            const uint64_t x = mul2(pair(z[h], z[h + 1]), mul2(twice(ks), pair(unit[h], unit[h + 1])));
            const uint64_t u = mul2(x, twice(p.scale_over_cap));
            const float2 in = both(u), low = capped_low(x, u, p.scale_log2e);
            z[h] = low.x, z[h + 1] = low.y;
            if (__any_sync(0xffffffffu, !(fabsf(in.x) < kBent && fabsf(in.y) < kBent))) {
              const float2 high = capped_high(u, p.cap_log2e);
              if (!(fabsf(in.x) < kBent)) z[h] = high.x;
              if (!(fabsf(in.y) < kBent)) z[h + 1] = high.y;
            }
          }
        } else {
          const float factor = ks * p.scale_log2e;
#pragma unroll
          for (int h = 0; h < HS; ++h) z[h] *= factor * unit[h];
        }
        if (slopes != nullptr) {
#pragma unroll
          for (int h = 0; h < HS; ++h) z[h] = fmaf((h < heads ? slopes[h] : 0.0f) * kLog2e, away, z[h]);
        }
        const float vs_least = fmaxf(fabsf(vs), kLeast), most = kLimit / vs_least;
        bool over = false;
#pragma unroll
        for (int h = 0; h < HS; ++h) over = over || exp2_fast(z[h] - ref[h]) > most;
        // where its weights go, those of p_bufs tiles ago have been used
        if (i >= S::p_bufs) {
          const int before = at - S::p_bufs;
          ok = wait_or_stop(&sh.pv_done[before & 7], (before >> 3) & 1, stop) && ok;
        }
        if (set_any(set, over && seen)) {
          // Move the references, by whole numbers, to leave the largest weight in (2^6, 2^7].
          const float more = log2f(vs_least);
#pragma unroll
          for (int h = 0; h < HS; ++h) {
            const float w = seen && z[h] == z[h] ? z[h] + more : __int_as_float(0xff800000);
            const int32_t m = __reduce_max_sync(0xffffffffu, ordered(w));
            if (lane == 0) sh.most[warp][h] = from_ordered(m);
          }
          set_sync(set);
          if (e < HS) {
            const float(*m)[HS] = &sh.most[set * 4];
            const float top = fmaxf(fmaxf(m[0][e], m[1][e]), fmaxf(m[2][e], m[3][e]));
            const float moved = fmaxf(ref[e], ceilf(top) - 7.0f);
            sh.factor[set * HS + e] = moved == ref[e] ? 1.0f : exp2_fast(ref[e] - moved);
            ref[e] = moved;
          }
          set_sync(set);
          const float* factor = sh.factor + set * HS;
#pragma unroll
          for (int h = 0; h < HS; ++h) sum[h] *= factor[h];
          if (i > 0) {
            ok = wait_or_stop(&sh.pv_done[(at - 1) & 7], ((at - 1) >> 3) & 1, stop) && ok;
            tc_fence_after();
            for (int m = 0; m < p.v_blocks; ++m)
#pragma unroll
              for (int t = 0; t < TERMS; ++t) {
                uint32_t v[HS];
                const uint32_t o_at = tmem_o + m * N + lanes + t * G + set * HS;
                tmem_ld(v, o_at);
                tmem_wait_ld(v);
#pragma unroll
                for (int h = 0; h < HS; ++h) v[h] = __float_as_uint(__uint_as_float(v[h]) * factor[h]);
                tmem_st(o_at, v);
              }
            tmem_wait_st();
          }
        }
        const uint32_t to = p_mine + (at % S::p_bufs) * (S::rows * 128) + set * HS * 128;
#pragma unroll
        for (int h = 0; h < HS; h += 2) {
          const float w0 = seen ? exp2_fast(z[h] - ref[h]) : 0.0f, w1 = seen ? exp2_fast(z[h + 1] - ref[h + 1]) : 0.0f;
          sum[h] += w0, sum[h + 1] += w1;
          uint32_t x = half_two(w0 * vs, w1 * vs);
#pragma unroll
          for (int t = 0; t < TERMS; ++t) {
            const uint32_t two = e4m3_of_half2(x);
            if (t + 1 < TERMS) x = rest16(x, half2_of_e4m3(two));
            // row t G + h of 128 bytes, in the swizzle: G and the set's first head are whole groups of 8 rows
            put_byte((to ^ ((h & 7) << 4)) + (t * G + h) * 128, two);
            put_byte((to ^ (((h + 1) & 7) << 4)) + (t * G + h + 1) * 128, two >> 8);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&sh.p_full[at & 7]);
        if (++note == p.notes) note = 0;
      }

      // ---- end of a work ----
      if (tiles > 0) ok = wait_or_stop(&sh.pv_done[(n + tiles - 1) & 7], ((n + tiles - 1) >> 3) & 1, stop) && ok;
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < HS; ++h) sum[h] = ok ? sum[h] : __int_as_float(0x7fc00000);
      const float part = sum_lanes<HS>(sum, lane);
      if (lane % (32 / HS) == 0) sh.sum[warp][lane / (32 / HS)] = part;
      set_sync(set);
      if (e < HS) {
        const float(*m)[HS] = &sh.sum[set * 4];
        const float total = (m[0][e] + m[1][e]) + (m[2][e] + m[3][e]);
        if (cluster > 1) {
          sh.head_ref[set * HS + e] = ref[e], sh.head_sum[set * HS + e] = total;
        } else {
          sh.inverse[set * HS + e] = e4_inverse(total);
          if (a.lse != nullptr && e < heads) a.lse[k.row * a.Hq + k.head0 + set * HS + e] = e4_logsum(ref[e], total);
        }
      }
      set_sync(set);
      const float* inverse = sh.inverse + set * HS;
      E* out = static_cast<E*>(a.out) + (k.row * a.Hq + k.head0 + set * HS) * a.Dv;
      const int pad = p.v_blocks * 128;
      float* rows = reinterpret_cast<float*>(smem) + set * HS * pad;
      for (int m = 0; m < p.v_blocks; ++m) {
        float x[HS];
#pragma unroll
        for (int h = 0; h < HS; ++h) x[h] = 0.0f;
        if (tiles > 0) {
          uint32_t v[TERMS][HS];
          const uint32_t o_at = tmem_o + m * N + lanes + set * HS;
#pragma unroll
          for (int t = 0; t < TERMS; ++t) tmem_ld(v[t], o_at + t * G);
#pragma unroll
          for (int t = 0; t < TERMS; ++t) tmem_wait_ld(v[t]);
#pragma unroll
          for (int h = 0; h < HS; ++h) {
            x[h] = __uint_as_float(v[TERMS - 1][h]);
#pragma unroll
            for (int t = TERMS - 2; t >= 0; --t) x[h] = fmaf(x[h], 0x1p-4f, __uint_as_float(v[t][h]));
          }
          if (m == p.v_blocks - 1) {  // O is read: the next work may have it
            tc_fence_before();
            mbar_arrive(&sh.o_free);
          }
        }
        const int d = m * 128 + e;
        if (cluster > 1) {
#pragma unroll
          for (int h = 0; h < HS; ++h) rows[h * pad + d] = x[h];
        } else if (d < a.Dv) {
#pragma unroll
          for (int h = 0; h < HS; ++h)
            if (h < heads) out[static_cast<int64_t>(h) * a.Dv + d] = E(x[h] * inverse[h]);
        }
      }
      set_sync(set);  // what the set shares is read
    }
  }

  __syncthreads();
  if (*stop != 0) {  // a wait ran out: nobody may have waited for what is in flight
    if (one) mma_drain(&sh.drained[warp - S::mma]);
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
      float m[8], l[8], all = kNothing, total = 0.0f;
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
  const int q_bytes = S::rows * 128 * p.d_blocks * S::q_bufs, p_bytes = S::rows * 128 * S::p_bufs;
  const int fixed = q_bytes + p_bytes + static_cast<int>(sizeof(Shared)) + kBufs * p.note_bytes;
  const int stage = p.k_bytes + p.v_bytes + p.note_bytes;
  const int join = G * p.v_blocks * 128 * 4;  // rows for the other CTAs, over the queries and the rings
  // Two CTAs share an SM where two stages each fit, else one has as many stages as fit.
  const int half = kMaxShared / 2 - 1024;
  const bool two = S::per_sm == 2 && fixed + 2 * stage <= half && p.tmem_cols <= 256 && join <= half - fixed + q_bytes;
  const int room = (two ? half : kMaxShared) - fixed;
  p.k_stages = room / stage < kMaxStages ? room / stage : kMaxStages;
  if (p.k_stages < 1) return TOPK_EINVAL;
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
  // Few rows: share each over the CTAs that would idle, down to two tiles each.
  const int64_t slots = static_cast<int64_t>(sm_count) * (two ? 2 : 1);
  const int tiles = a.K / kEntries + (a.K % kEntries != 0);
  int cluster = 1;
  while (cluster < 8 && work * cluster * 2 <= slots && cluster * 4 <= tiles) cluster *= 2;
  const int64_t grid = cluster == 1 && work > slots ? slots : work * cluster;
  if ((work / grid + 1) * tiles > INT32_MAX) return TOPK_EINVAL;  // a CTA counts its tiles
  constexpr auto kernel = cache_attention_kernel<E, G>;
  const topk_status st = allow_shared<kernel>(dev);
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

// The least padded heads that hold those of a key head, or tiles of the most.
template <typename E>
topk_status launch_cache_attention(const sparse_attention_e4m3_args& a, int dev, int sm_count, cudaStream_t stream) {
  const int heads = a.attention.Hq / a.attention.Hkv;
  if (heads <= 8) return launch_heads<E, 8>(a, dev, sm_count, stream);
  if (heads <= 16) return launch_heads<E, 16>(a, dev, sm_count, stream);
  // Three terms of 64 heads would not leave TMEM for their scores.
  if (heads <= 32 || !std::is_same<E, __nv_bfloat16>::value) return launch_heads<E, 32>(a, dev, sm_count, stream);
  if constexpr (std::is_same<E, __nv_bfloat16>::value) return launch_heads<E, 64>(a, dev, sm_count, stream);
  return TOPK_EINVAL;
}

}  // namespace
}  // namespace tki
