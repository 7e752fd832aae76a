// Indexer scores over a paged key cache (include/sparse_step.h,
// sparse_indexer_scores).
//
//   out[b, t, s] = ks[s] sum_h w[b, t, h] max(0, q[b, t, h] . k[s])
//
// The products run on the tensor cores with the keys as the rows: a tile of
// 128 positions (TMEM lanes) by the heads of up to 32 query tokens (columns,
// 256 at most). So one thread of the epilogue holds all the products of one
// position, and the sum over heads needs no exchange: a maximum and a
// multiply-add per product (packed multiply-adds cost a move each, 4.6
// instructions a product in all; the accumulator's own layout, which needs a
// quarter of the weights per thread, reads TMEM slower: half as long again). A
// tile of keys is fetched once for all query tokens of its group.
//
// One CTA per SM, 20 warps: three fetch (keys through the page table into a
// ring, by TMA boxes or, where pages are too odd for them, 16-byte copies;
// zeros for absent rows and the padding of D; queries and weights of the next
// work unit), one thread issues the products into two TMEM buffers, sixteen
// warps sum over heads. Work units are (sequence, range of tiles, group of
// query tokens).
//
// Measured: decode, 64 sequences of up to 65536 positions, 64 heads, bf16, 155
// us, 6.3 TB/s (145 us for its bytes at the measured copy rate): HBM bound.
// Prefill, 2048 tokens on 8192 positions, 165 us, 1.5 PFLOP/s (127 us at
// the measured matrix rate): the tensor pipe is busy in 66 % of the cycles and
// the issue slots in 67 %; with two TMEM buffers products wait for a buffer's
// whole read and sums for a whole product. e4m3, 32 sequences x 2 tokens x 32769,
// pages of 16, 40 us (20): HBM at 39 %, the tensor pipe at 9 %; every role makes
// a round of waits for each tile, which is half the bytes of a 16-bit one.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "step_launch.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace tki {
namespace {

constexpr int kTile = 128;             // positions per tile: the rows of one product
constexpr int kEpilogueWarps = 16;
constexpr int kFetchWarp = kEpilogueWarps, kProductWarp = kFetchWarp + 3;
constexpr int kScoreThreads = (kProductWarp + 1) * 32;
constexpr int kMaxTokens = 32;         // query tokens per group
constexpr int kMaxCols = 256;

struct ScoreParams {
  sparse_scores_args a;
  int32_t hp;              // heads of a token, padded to 8, 16, 32, 64 or 128
  int32_t hp_shift;        // its logarithm
  int32_t tokens;          // query tokens per group
  int32_t cols;            // tokens * hp
  int32_t blocks;          // 128-byte blocks per key: 1 or 2
  int32_t row_units;       // 16-byte units of D
  int32_t unit_tiles;      // tiles per work unit
  int32_t share;           // groups of epilogue warps per tile: 1 or 2
  int32_t page_shift;      // log2 of page_size, or -1
  uint32_t pages;
  int32_t chunks, groups;  // work units per sequence: chunks x groups
  uint32_t units;
  bool q_boxes;            // queries come by the TMA engine ...
  bool q_vector;           // ... or 16 bytes at a time, else element by element
  int32_t box_rows;        // entries of one page per box of the keys' map, 0 without one
  CUtensorMap map, q_map;
};

// A work unit: sequence, first query token and their number, range of tiles.
struct Unit {
  int b, t0, tokens, tile0, tile1;
};

struct ScoreShared {
  alignas(16) float weights[2][kMaxCols];  // read four at a time
  int32_t lengths[2][kMaxTokens];
  uint64_t full[6], q_full[2], q_empty[2];
  uint64_t t_full[8], t_empty[8];  // of tile k at k % 8: nobody who waits on one lags behind by eight tiles
  uint64_t drained;
  Unit units[2];  // with the queries; no tiles: the end
  uint32_t tmem;
  uint32_t stop;
};

__device__ __forceinline__ int length_of(const ScoreParams& p, int b, int t) {
  const int n = p.a.lengths[static_cast<int64_t>(b) * p.a.T + t];
  return n < 0 ? 0 : min(static_cast<int64_t>(n), p.a.width);
}

__device__ __forceinline__ Unit unit_of(const ScoreParams& p, uint32_t u) {
  Unit r;
  const uint32_t c = u / static_cast<uint32_t>(p.groups);
  r.t0 = static_cast<int>(u - c * p.groups) * p.tokens;
  r.b = static_cast<int>(c / static_cast<uint32_t>(p.chunks));
  r.tokens = min(p.tokens, p.a.T - r.t0);
  const int lane = threadIdx.x & 31;
  const int longest = __reduce_max_sync(0xffffffffu, lane < r.tokens ? length_of(p, r.b, r.t0 + lane) : 0);
  r.tile0 = static_cast<int>(c - static_cast<uint32_t>(r.b) * p.chunks) * p.unit_tiles;
  r.tile1 = min(r.tile0 + p.unit_tiles, longest / kTile + (longest % kTile != 0));
  return r;
}

__device__ __forceinline__ uint32_t page_index(const ScoreParams& p, uint32_t s) {
  return p.page_shift >= 0 ? s >> p.page_shift : s / static_cast<uint32_t>(p.a.page_size);
}
__device__ __forceinline__ uint32_t place_in_page(const ScoreParams& p, uint32_t s) {
  return s - page_index(p, s) * static_cast<uint32_t>(p.a.page_size);
}
// The page id of position s of a sequence, ~0 (no page) from `end` on.
__device__ __forceinline__ uint32_t page_at(const ScoreParams& p, const int32_t* table, uint32_t s, uint32_t end) {
  return s < end ? static_cast<uint32_t>(table[page_index(p, s)]) : 0xffffffffu;
}

// max(0, x), a NaN kept. Volatile: it stays behind the wait for the products.
__device__ __forceinline__ float relu(uint32_t x) {
  float r;
  asm volatile("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(__uint_as_float(x)));
  return r;
}

template <typename E>
struct Kind;
template <>
struct Kind<__nv_bfloat16> {
  static constexpr uint32_t type = 1;
  static constexpr CUtensorMapDataType map_type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
};
template <>
struct Kind<__half> {
  static constexpr uint32_t type = 0;
  static constexpr CUtensorMapDataType map_type = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
};
template <>
struct Kind<__nv_fp8_e4m3> {
  static constexpr uint32_t type = 0;
  static constexpr CUtensorMapDataType map_type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
};

// Queries, weights and lengths of a unit into buffer `buf`, by N threads, each
// of which arrives twice on q_full.
template <typename E, int N>
__device__ __forceinline__ void fetch_queries(const ScoreParams& p, const Unit& r, unsigned char* smem, uint32_t q_bytes,
                                              ScoreShared& sh, uint32_t buf, int th, const void* nowhere) {
  if (p.q_boxes) {
    if (th == 0) {
      mbar_arrive_expect_tx(&sh.q_full[buf], q_bytes);
      for (int c = 0; c < p.blocks; ++c)
        box_load(smem_addr(smem) + buf * q_bytes + c * p.cols * 128, &p.q_map, c * (128 / static_cast<int>(sizeof(E))), 0,
                 r.t0, r.b, &sh.q_full[buf]);
    } else {
      mbar_arrive(&sh.q_full[buf]);
    }
  } else {
    const int unit16 = th & 7;
    for (int t = 0; t < p.tokens; ++t)
      for (int h = th >> 3; h < p.hp; h += N / 8) {
        const E* q = static_cast<const E*>(p.a.q) + r.b * p.a.q_seq_stride + (r.t0 + t) * p.a.q_token_stride +
                     h * p.a.q_head_stride;
        for (int c = 0; c < p.blocks; ++c) {
          const int j = c * 8 + unit16;
          const bool real = t < r.tokens && h < p.a.H && j < p.row_units;
          const E* src = q + j * (16 / sizeof(E));
          const uint32_t at = buf * q_bytes + c * p.cols * 128 + swizzled(t * p.hp + h, unit16);
          if (p.q_vector) {
            copy16(smem_addr(smem) + at, real ? src : nowhere, real);
          } else {
            alignas(16) E v[16 / sizeof(E)];
            for (int e = 0; e < static_cast<int>(16 / sizeof(E)); ++e) v[e] = real ? src[e] : E(0.0f);
            *reinterpret_cast<uint4*>(smem + at) = *reinterpret_cast<const uint4*>(v);
          }
        }
      }
    copy_arrive(&sh.q_full[buf]);
  }
  const float* w = p.a.weights + (static_cast<int64_t>(r.b) * p.a.T + r.t0) * p.a.H;
  for (int first = th; first < p.cols; first += 4 * N) {  // four reads in flight
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = first + u * N, t = i >> p.hp_shift, h = i & (p.hp - 1);
      v[u] = t < r.tokens && h < p.a.H ? w[t * p.a.H + h] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (first + u * N < p.cols) sh.weights[buf][first + u * N] = v[u];
  }
  if (th < kMaxTokens) sh.lengths[buf][th] = th < r.tokens ? length_of(p, r.b, r.t0 + th) : 0;
  if (th == 0) sh.units[buf] = r;
  mbar_arrive(&sh.q_full[buf]);
}

// No copy may arrive after the CTA has left.
__device__ __forceinline__ void queries_arrived(ScoreShared& sh, uint32_t nu) {
  for (uint32_t i = 0; i < 2 && i < nu; ++i)
    mbar_wait_bounded(&sh.q_full[(nu - 1 - i) & 1], ((nu - 1 - i) >> 1) & 1, 1000000000ull);
  copy_commit();
  copy_wait<0>();
}

// The scores of one (present) position for query tokens [t0, t1) of a unit,
// product by product over the heads alone.
template <typename E>
__device__ __noinline__ void score_again(const ScoreParams& p, const ScoreShared& sh, uint32_t buf, int t0, int t1, uint32_t s) {
  const Unit& r = sh.units[buf];
  const uint32_t page = static_cast<uint32_t>(p.a.page_table[r.b * p.a.table_stride + page_index(p, s)]);
  const uint32_t place = place_in_page(p, s);
  const E* key = static_cast<const E*>(p.a.keys) + page * p.a.key_page_stride + place * p.a.key_token_stride;
  const float scale = p.a.key_scales != nullptr ? p.a.key_scales[static_cast<int64_t>(page) * p.a.page_size + place] : 1.0f;
  for (int t = t0; t < t1; ++t) {
    if (s >= static_cast<uint32_t>(sh.lengths[buf][t])) continue;
    const E* q = static_cast<const E*>(p.a.q) + r.b * p.a.q_seq_stride + (r.t0 + t) * p.a.q_token_stride;
    float sum = 0.0f;
    for (int h = 0; h < p.a.H; ++h, q += p.a.q_head_stride) {
      float dot = 0.0f;
      for (int d = 0; d < p.a.D; ++d) dot = fmaf(static_cast<float>(q[d]), static_cast<float>(key[d]), dot);
      sum = fmaf(sh.weights[buf][t * p.hp + h], relu(__float_as_uint(dot)), sum);
    }
    p.a.out[r.b * p.a.out_seq_stride + (r.t0 + t) * p.a.out_token_stride + s] = sum * scale;
  }
}

// STAGES tiles of keys in flight; HP columns a token; keys by BOXES of
// the TMA engine or by 16-byte copies.
template <typename E, int STAGES, int HP, bool BOXES>
__global__ void __launch_bounds__(kScoreThreads, 1) scores_kernel(const __grid_constant__ ScoreParams p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t q_bytes = static_cast<uint32_t>(p.cols) * 128 * p.blocks;
  const uint32_t tile_bytes = kTile * 128 * p.blocks;
  unsigned char* ring = smem + 2 * q_bytes;
  ScoreShared& sh = *reinterpret_cast<ScoreShared*>(ring + STAGES * tile_bytes);
  const uint32_t q_addr = smem_addr(smem), ring_addr = smem_addr(ring);

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&sh.full[i], BOXES ? 1 : 64);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], BOXES ? 128 : 64);  // two of each fetching thread
      mbar_init(&sh.q_empty[i], 1 + kEpilogueWarps);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&sh.t_full[i], 1), mbar_init(&sh.t_empty[i], 128 * p.share);
    mbar_init(&sh.drained, 1);
    sh.stop = 0;
    fence_mbar_init();
  }
  if (warp == kProductWarp) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile uint32_t* stop = &sh.stop;
  bool one = false;  // the thread that issues products

  // what a copy of nothing points at
  const void* nowhere = reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(p.a.q) & ~static_cast<uintptr_t>(15));
  if (BOXES && warp == kFetchWarp) {
    // ---- keys, by boxes: lane i fetches block i / 16 of the box i % 16 of a tile ----
    const int box = lane & 15, block = lane >> 4, boxes = kTile / p.box_rows;
    const bool mine = box < boxes && block < p.blocks;
    // The next unit's length and first page ids are read while this one's
    // boxes are under way.
    uint32_t k = 0, u = blockIdx.x, at = 0, end = 0, next = 0;
    const int32_t* table = nullptr;
    Unit r = {};
    auto advance = [&]() {  // to the next unit with work, its first lookup made
      for (r.tile1 = 0, r.tile0 = 0; u < p.units; u += gridDim.x) {
        r = unit_of(p, u);
        if (r.tile0 < r.tile1) break;
      }
      if (r.tile0 >= r.tile1) return;
      u += gridDim.x;
      table = p.a.page_table + r.b * p.a.table_stride;
      end = mine ? min(static_cast<uint32_t>(r.tile1) * kTile, static_cast<uint32_t>(p.a.width)) : 0;
      at = static_cast<uint32_t>(r.tile0) * kTile + box * p.box_rows;  // of the lane's box
      next = page_at(p, table, at, end);
    };
    advance();
    int tiles = r.tile1 - r.tile0;
    bool ok = true;
    while (tiles > 0 && ok) {
      int tiles_after = 0;
      for (int i = 0; i < tiles; ++i, ++k) {
        const uint32_t stage = k % STAGES, page = next, here = at;
        if (i + 1 < tiles) {  // a tile ahead
          at += kTile;
          next = page_at(p, table, at, end);
        } else {
          advance();
          tiles_after = r.tile1 - r.tile0;
        }
        ok = k < STAGES || wait_or_stop(&sh.t_full[(k - STAGES) & 7], ((k - STAGES) >> 3) & 1, stop);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[stage], tile_bytes);
        __syncwarp();
        if (mine) {
          const int z = static_cast<int>(min(page, p.pages));  // absent: outside, zeros
          const int y = static_cast<int>(place_in_page(p, here));
          box_load(ring_addr + stage * tile_bytes + (block * kTile + box * p.box_rows) * 128, &p.map,
                   block * (128 / static_cast<int>(sizeof(E))), y, z, &sh.full[stage]);
        }
      }
      tiles = tiles_after;
    }
    // no box may arrive after the CTA has left
    for (uint32_t i = 0; i < STAGES && i < k; ++i)
      mbar_wait_bounded(&sh.full[(k - 1 - i) % STAGES], ((k - 1 - i) / STAGES) & 1, 1000000000ull);
  } else if (!BOXES && (warp == kFetchWarp || warp == kFetchWarp + 1)) {
    // ---- keys, by 16-byte copies: 8 lanes fetch a row's 128 bytes ----
    const int w = warp - kFetchWarp;
    const uint32_t unit16 = lane & 7, sub = lane >> 3;
    const E* keys = static_cast<const E*>(p.pages > 0 ? p.a.keys : nowhere);  // an empty cache has no address
    uint32_t k = 0;
    bool ok = true;
    for (uint32_t u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
      const Unit r = unit_of(p, u);
      if (r.tile0 >= r.tile1) continue;
      const int32_t* table = p.a.page_table + r.b * p.a.table_stride;
      const uint32_t end = min(static_cast<uint32_t>(r.tile1) * kTile, static_cast<uint32_t>(p.a.width));
      // this lane looks up rows 64 w + lane and 64 w + 32 + lane of a tile
      uint32_t at = static_cast<uint32_t>(r.tile0) * kTile + w * 64 + lane;
      uint32_t next[2] = {page_at(p, table, at, end), page_at(p, table, at + 32, end)};  // read a tile ahead
      for (int tile = r.tile0; tile < r.tile1; ++tile, ++k, at += kTile) {
        const uint32_t stage = k % STAGES;
        const uint32_t page[2] = {next[0], next[1]};
        next[0] = page_at(p, table, at + kTile, end);
        next[1] = page_at(p, table, at + kTile + 32, end);
        ok = k < STAGES || wait_or_stop(&sh.t_full[(k - STAGES) & 7], ((k - STAGES) >> 3) & 1, stop);
        if (!ok) break;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const bool here = page[half] < p.pages;
          const uint32_t bits = __ballot_sync(0xffffffffu, here);
          const int64_t slot = here ? page[half] * p.a.key_page_stride +
                                          place_in_page(p, at + 32 * half) * p.a.key_token_stride
                                    : 0;
          const uint32_t dst = ring_addr + stage * tile_bytes + (w * 64 + half * 32 + sub) * 128;
          const E* from[8];
          uint32_t bytes[8];  // to copy: none of an absent entry
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            from[i] = keys + __shfl_sync(0xffffffffu, slot, 4 * i + sub);
            bytes[i] = (bits >> (4 * i + sub)) & 1 ? 16 : 0;
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (c >= p.blocks) break;
            const uint32_t j = c * 8 + unit16;
            const bool inside = j < static_cast<uint32_t>(p.row_units);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t at = c * kTile * 128 + i * 512 + ((unit16 ^ (sub + 4 * (i & 1))) << 4);
              copy_bytes(dst + at, inside ? static_cast<const void*>(from[i] + j * (16 / sizeof(E))) : nowhere,
                         inside ? bytes[i] : 0);
            }
          }
        }
        copy_arrive(&sh.full[stage]);
      }
    }
    copy_commit();
    copy_wait<0>();
  } else if (warp >= kFetchWarp && warp < kProductWarp) {
    // ---- queries, a unit ahead ----
    constexpr int kFirst = kFetchWarp + (BOXES ? 1 : 2);
    uint32_t nu = 0;
    for (uint32_t u = blockIdx.x; u < p.units; u += gridDim.x) {
      const Unit r = unit_of(p, u);
      if (r.tile0 >= r.tile1) continue;
      if (!wait_or_stop(&sh.q_empty[nu & 1], ((nu >> 1) & 1) ^ 1, stop)) break;
      fetch_queries<E, (kProductWarp - kFirst) * 32>(p, r, smem, q_bytes, sh, nu & 1, threadIdx.x - kFirst * 32, nowhere);
      ++nu;
    }
    if (wait_or_stop(&sh.q_empty[nu & 1], ((nu >> 1) & 1) ^ 1, stop)) {  // the end
      if (threadIdx.x == kFirst * 32) sh.units[nu & 1] = Unit{};
      mbar_arrive(&sh.q_full[nu & 1]);
      mbar_arrive(&sh.q_full[nu & 1]);
      ++nu;
    }
    queries_arrived(sh, nu);
  } else if (warp == kProductWarp) {
    // ---- products ----
    const uint32_t desc = mma_desc(Kind<E>::type, p.cols);
    const uint64_t ring_desc = operand_desc(ring_addr), q_desc = operand_desc(q_addr);
    uint32_t k = 0, stage = 0, turn = 0;
    bool ok = true;
    one = elect_one();
    for (uint32_t nu = 0; ok; ++nu) {
      const uint32_t buf = nu & 1;
      ok = wait_or_stop(&sh.q_full[buf], (nu >> 1) & 1, stop);
      if (!ok) break;
      const Unit r = sh.units[buf];
      if (r.tile0 >= r.tile1) break;
      if (!p.q_boxes) fence_proxy_async_smem();  // copies and stores are in; now the tensor cores may see them
      // one thread from here: its waits need no vote
      const int tiles = r.tile1 - r.tile0;
      bool done = true;
      if (one) {
        const uint64_t db = q_desc + (buf * q_bytes >> 4);
        uint32_t st = stage, tn = turn;
        for (int i = 0; i < tiles; ++i) {
          const uint32_t kk = k + i, to = tmem + (kk & 1) * kMaxCols;
          // the buffer is free when tile k - 2 is read
          done = (kk < 2 || wait_or_stop_one(&sh.t_empty[(kk - 2) & 7], ((kk - 2) >> 3) & 1, stop)) &&
                 wait_or_stop_one(&sh.full[st], tn, stop);
          if (!done) break;
          if (!BOXES) fence_proxy_async_smem();
          tc_fence_after();
          const uint64_t da = ring_desc + (st * tile_bytes >> 4);
          for (int c = 0; c < p.blocks; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint64_t a = da + static_cast<uint32_t>(c * (kTile * 128 >> 4) + j * 2);
              const uint64_t b = db + static_cast<uint32_t>(c * (p.cols * 128 >> 4) + j * 2);
              if constexpr (sizeof(E) == 1)
                mma_f8(to, a, b, desc, c + j > 0);
              else
                mma_f16(to, a, b, desc, c + j > 0);
            }
          mma_commit(&sh.t_full[kk & 7]);
          if (++st == STAGES) st = 0, tn ^= 1;
        }
        if (done) mma_commit(&sh.q_empty[buf]);
      }
      __syncwarp();
      ok = __all_sync(0xffffffffu, done);
      k += tiles;
      stage += tiles % STAGES;
      if (((tiles / STAGES) & 1) != 0) turn ^= 1;
      if (stage >= STAGES) stage -= STAGES, turn ^= 1;
    }
  } else {
    // ---- sums over heads ----
    // Four groups of four warps, each with all 128 positions of a tile: two
    // share every other tile's tokens, or, where there is one token, each takes
    // every fourth tile. (2048 x 8192: 165 us by two; by one 188, by all four,
    // which then wait and sum in step, 198. Two tokens, e4m3: 39.9 by two, 38.5 by one.)
    const int group = warp >> 2, quarter = warp & 3;
    const int tile_step = 4 / p.share, turn_of = group / p.share, part = group % p.share;
    const uint32_t lanes = static_cast<uint32_t>(quarter) << 21;
    uint32_t k = 0;
    bool ok = true;
    for (uint32_t nu = 0; ok; ++nu) {
      const uint32_t buf = nu & 1;
      ok = wait_or_stop(&sh.q_full[buf], (nu >> 1) & 1, stop);
      if (!ok) break;
      const Unit r = sh.units[buf];
      if (r.tile0 >= r.tile1) break;
      constexpr int kPer = HP < 32 ? 32 / HP : 1;  // tokens in 32 columns, which are not split
      const int packs = (r.tokens + kPer - 1) / kPer;
      const int t_first = packs * part / p.share * kPer, t1 = min(packs * (part + 1) / p.share * kPer, r.tokens);
      float* out = p.a.out + r.b * p.a.out_seq_stride + (r.t0 + t_first) * p.a.out_token_stride;
      const int32_t* table = p.a.page_table + r.b * p.a.table_stride;
      const uint32_t end = min(static_cast<uint32_t>(r.tile1) * kTile, static_cast<uint32_t>(p.a.width));
      const uint32_t skip = static_cast<uint32_t>(turn_of - static_cast<int>(k)) & (tile_step - 1);
      const int mine = r.tile0 + static_cast<int>(skip);
      uint32_t s = static_cast<uint32_t>(mine) * kTile + quarter * 32 + lane;
      uint32_t next = page_at(p, table, s, end);
      const uint32_t k0 = k;
      k += skip;
      for (int tile = mine; tile < r.tile1; tile += tile_step, k += tile_step, s += tile_step * kTile) {
        const uint32_t page = next;
        next = page_at(p, table, s + tile_step * kTile, end);
        const bool absent = page >= p.pages;
        float scale = 1.0f;
        if (!absent && p.a.key_scales != nullptr)
          scale = p.a.key_scales[static_cast<int64_t>(page) * p.a.page_size + place_in_page(p, s)];
        const uint32_t tb = k & 1;
        ok = wait_or_stop(&sh.t_full[k & 7], (k >> 3) & 1, stop);
        if (!ok) break;
        tc_fence_after();
        int left = HP < 32 ? (t1 - t_first + kPer - 1) / kPer : (t1 - t_first) * (HP / 32);  // times 32 columns
        if (left <= 0) {
          mbar_arrive(&sh.t_empty[k & 7]);
          continue;
        }
        uint32_t at = tmem + tb * kMaxCols + lanes + t_first * HP;
        const float* wt = sh.weights[buf] + t_first * HP;
        const int32_t* length = sh.lengths[buf] + t_first;
        float* o = out + s;
        float acc[4] = {};
        uint32_t v0[32], v1[32];
        auto release = [&]() {  // the buffer is read: the next product may have it
          tc_fence_before();
          mbar_arrive(&sh.t_empty[k & 7]);
        };
        auto add = [&](const uint32_t (&v)[32], const float* w) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 ww = *reinterpret_cast<const float4*>(w + j);
            acc[0] = fmaf(ww.x, relu(v[j]), acc[0]);
            acc[1] = fmaf(ww.y, relu(v[j + 1]), acc[1]);
            acc[2] = fmaf(ww.z, relu(v[j + 2]), acc[2]);
            acc[3] = fmaf(ww.w, relu(v[j + 3]), acc[3]);
          }
        };
        float sum = 0.0f;  // of the last token
        auto finish = [&]() {
          sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
          if (s < static_cast<uint32_t>(*length)) *o = absent ? __int_as_float(0xff800000) : sum * scale;
          acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
          ++length, o += p.a.out_token_stride;
        };
        int tokens = t1 - t_first;
        // 32 columns that hold several tokens
        auto add_all = [&](const uint32_t (&v)[32], const float* w) {
#pragma unroll
          for (int g = 0; g < kPer; ++g) {
            if (g >= tokens) break;
#pragma unroll
            for (int j = 0; j < 32 / kPer; j += 4) {
              const int e = g * (32 / kPer) + j;
              const float4 ww = *reinterpret_cast<const float4*>(w + e);
              acc[0] = fmaf(ww.x, relu(v[e]), acc[0]);
              acc[1] = fmaf(ww.y, relu(v[e + 1]), acc[1]);
              acc[2] = fmaf(ww.z, relu(v[e + 2]), acc[2]);
              acc[3] = fmaf(ww.w, relu(v[e + 3]), acc[3]);
            }
            finish();
          }
          tokens -= kPer;
        };
        for (; left > 0; left -= 2, at += 64, wt += 64) {
          const bool both = HP > 32 || left > 1;
          tmem_ld(v0, at);
          if (both) tmem_ld(v1, at + 32);
          tmem_wait_ld();
          if (left <= 2) release();
          if constexpr (HP <= 32) {
            add_all(v0, wt);
            if (both) add_all(v1, wt + 32);
          } else {
            add(v0, wt);
            add(v1, wt + 32);
            if (HP < 128 || (left & 2) != 0) finish();
          }
        }
        // A key that is not finite makes NaN of the zeros of a head that is
        // only padding, in every token's sum, which the formula has not: such
        // a position is summed again. (Padded columns left out of all sums
        // instead: 2048 x 8192, 64 heads, 174 us for 164; 1024 x 8192, 24 heads, 72 for 61.)
        if (sizeof(E) > 1 && sum != sum && !absent && p.a.H < HP) score_again<E>(p, sh, buf, t_first, t1, s);
      }
      k = k0 + (r.tile1 - r.tile0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_empty[buf]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*stop != 0) {  // a wait ran out: NaN, not half a result
    if (one) mma_drain(&sh.drained);
    __syncwarp();
    for (uint32_t u = blockIdx.x; u < p.units; u += gridDim.x) {
      const Unit r = unit_of(p, u);
      for (int t = 0; t < r.tokens; ++t) {
        const int64_t end = min(static_cast<int64_t>(r.tile1) * kTile, static_cast<int64_t>(length_of(p, r.b, r.t0 + t)));
        for (int64_t s = static_cast<int64_t>(r.tile0) * kTile + threadIdx.x; s < end; s += kScoreThreads)
          p.a.out[r.b * p.a.out_seq_stride + (r.t0 + t) * p.a.out_token_stride + s] = __int_as_float(0x7fc00000);
      }
    }
  }
  if (warp == kProductWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

template <typename E, int STAGES, int HP, bool BOXES>
topk_status launch_variant(const ScoreParams& p, int dev, int sm_count, cudaStream_t stream) {
  static_assert(sizeof(ScoreShared) <= 3072 && offsetof(ScoreShared, weights) == 0, "behind the ring, aligned with it");
  const size_t bytes = 2 * static_cast<size_t>(p.cols) * 128 * p.blocks + STAGES * static_cast<size_t>(kTile) * 128 * p.blocks +
                       sizeof(ScoreShared);
  constexpr auto kernel = scores_kernel<E, STAGES, HP, BOXES>;
  const topk_status st = allow_shared<kernel>(dev);
  if (st != TOPK_OK) return st;
  const unsigned grid = p.units < static_cast<unsigned>(sm_count) ? p.units : static_cast<unsigned>(sm_count);
  return launch(kernel, p, dim3(grid), kScoreThreads, bytes, stream);
}

template <typename E, int STAGES, int HP>
topk_status launch_step(const ScoreParams& p, int dev, int sm_count, cudaStream_t stream) {
  return p.box_rows > 0 ? launch_variant<E, STAGES, HP, true>(p, dev, sm_count, stream)
                        : launch_variant<E, STAGES, HP, false>(p, dev, sm_count, stream);
}

template <typename E, int HP>
topk_status launch_ring(const ScoreParams& p, int dev, int sm_count, cudaStream_t stream) {
  // The ring gets what the queries leave of 227 KB: 6, 5 or 3 tiles.
  if (p.cols <= 64) return launch_step<E, 6, HP>(p, dev, sm_count, stream);
  if (p.cols <= 128) return launch_step<E, 5, HP>(p, dev, sm_count, stream);
  return launch_step<E, 3, HP>(p, dev, sm_count, stream);
}

template <typename E>
topk_status launch_scores_of(const sparse_scores_args& a, int dev, int sm_count, cudaStream_t stream) {
  ScoreParams p = {};
  p.a = a;
  const int size = sizeof(E);
  p.hp = a.H <= 8 ? 8 : a.H <= 16 ? 16 : a.H <= 32 ? 32 : a.H <= 64 ? 64 : 128;
  p.hp_shift = p.hp == 8 ? 3 : p.hp == 16 ? 4 : p.hp == 32 ? 5 : p.hp == 64 ? 6 : 7;
  // Tokens per group: 256 columns of them at most, in whole 32 columns.
  const int per = p.hp < 32 ? 32 / p.hp : 1;
  p.tokens = kMaxCols / p.hp;
  if (p.tokens > a.T) p.tokens = (a.T + per - 1) / per * per;
  p.cols = p.tokens * p.hp;
  p.blocks = (a.D * size + 127) / 128;
  p.row_units = a.D * size / 16;
  p.share = p.tokens >= 2 * per ? 2 : 1;
  p.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page_size == 1 << i) p.page_shift = i;
  p.pages = a.num_pages < INT32_MAX ? static_cast<uint32_t>(a.num_pages) : INT32_MAX;
  p.groups = a.T / p.tokens + (a.T % p.tokens != 0);
  // Work units of at most 16 tiles, 8 where a tile is short work: enough of
  // them to even out the SMs, long enough to hide the next unit's queries
  // (64 x 65536, 64 columns: 155.5 us by 8, 159 by 16; e4m3, 32 x 2 x 32769, 64
  // columns: 40.0 and 43.4; e4m3, 8 x 8 x 32769, 256 columns: 19.5 and 17.4. Two bytes and
  // 256 columns go either way: 2048 x 8192 161 by 8 and 164.5 by 16 with 64 heads, 323 and
  // 310 with 128); fewer while SMs would idle.
  const int most = p.cols <= 128 ? 8 : 16;
  const int64_t tiles = (a.width + kTile - 1) / kTile;
  if (tiles * p.groups > (INT64_MAX - sm_count) / a.B) return TOPK_EINVAL;
  const int64_t all = tiles * p.groups * a.B;
  const int64_t even = (all + sm_count - 1) / sm_count;
  p.unit_tiles = static_cast<int32_t>(even < most ? even : most);
  p.chunks = static_cast<int32_t>((tiles + p.unit_tiles - 1) / p.unit_tiles);
  const int64_t units = static_cast<int64_t>(p.chunks) * p.groups * a.B;
  if (units > INT32_MAX) return TOPK_EINVAL;
  p.units = static_cast<uint32_t>(units);
  p.q_vector = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && a.q_seq_stride * size % 16 == 0 &&
               a.q_token_stride * size % 16 == 0 && a.q_head_stride * size % 16 == 0;
  // Boxes hold entries of one page: the largest power of two that divides the
  // page, where it is at least 16 (64 x 65536: pages of 16 181 us by boxes, 199 by
  // copies; of 48 211 and 252; of 8 273 and 199).
  int rows = a.page_size & -a.page_size;
  rows = rows < kTile ? rows : kTile;
  const int64_t extents[3] = {a.D, a.page_size, a.num_pages}, strides[2] = {a.key_token_stride, a.key_page_stride};
  const int box[2] = {rows, 1};
  p.box_rows = rows >= 16 && box_map(&p.map, Kind<E>::map_type, size, a.keys, 3, extents, strides, box) ? rows : 0;
  // A unit's queries are one box more; heads and tokens that are not there
  // read as zeros.
  const int64_t q_extents[4] = {a.D, a.H, a.T, a.B}, q_strides[3] = {a.q_head_stride, a.q_token_stride, a.q_seq_stride};
  const int q_box[3] = {p.hp, p.tokens, 1};
  p.q_boxes = box_map(&p.q_map, Kind<E>::map_type, size, a.q, 4, q_extents, q_strides, q_box);
  if (p.hp == 8) return launch_ring<E, 8>(p, dev, sm_count, stream);
  if (p.hp == 16) return launch_ring<E, 16>(p, dev, sm_count, stream);
  if (p.hp == 32) return launch_ring<E, 32>(p, dev, sm_count, stream);
  if (p.hp == 64) return launch_ring<E, 64>(p, dev, sm_count, stream);
  return launch_ring<E, 128>(p, dev, sm_count, stream);
}

}  // namespace
}  // namespace tki
