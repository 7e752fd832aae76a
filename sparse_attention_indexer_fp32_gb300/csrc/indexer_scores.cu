// Indexer scores over a paged key cache (include/sparse_step.h,
// sparse_indexer_scores).
//
//   out[b, t, s] = ks[s] sum_h w[b, t, h] max(0, q[b, t, h] . k[s])
//
// The products run on the tensor cores with the keys as the rows: a tile of
// 128 positions (TMEM lanes) by the heads of up to 16 query tokens (columns,
// 256 at most). So one thread of the epilogue holds all the products of one
// position, and the sum over heads needs no exchange: a maximum and half a
// packed multiply-add per product. A tile of keys is fetched once for all
// query tokens of its group.
//
// One CTA per SM, 13 warps: four fetch keys through the page table into a
// ring (16-byte asynchronous copies, zeros for absent rows and for the
// padding of D), one thread issues the products into two TMEM buffers, two
// groups of four warps take the buffers in turn. Work units are (sequence,
// range of tiles, group of query tokens); queries, weights and lengths of the
// next unit are fetched while this one runs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "step_launch.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace tki {
namespace {

constexpr int kTile = 128;             // positions per tile: the rows of one product
constexpr int kScoreThreads = 13 * 32;
constexpr int kEpilogueWarps = 8;
constexpr int kMaxTokens = 16;         // query tokens per group
constexpr int kMaxCols = 256;

struct ScoreParams {
  sparse_scores_args a;
  int32_t hp;              // heads of a token, padded to whole column steps
  int32_t tokens;          // query tokens per group
  int32_t cols;            // tokens * hp
  int32_t blocks;          // 128-byte blocks per key: 1 or 2
  int32_t row_units;       // 16-byte units of D
  int32_t unit_tiles;      // tiles per work unit
  int32_t chunks, groups;  // work units per sequence: chunks x groups
  int64_t units;
  bool q_vector;           // queries can be fetched 16 bytes at a time
  int32_t box_rows;        // entries of one page per box of the tensor map
  CUtensorMap map;         // of the keys, where boxes are used
};

struct ScoreShared {
  float weights[2][kMaxCols];
  int32_t lengths[2][kMaxTokens];
  uint64_t full[6], empty[6], q_full[2], q_empty[2], t_full[2], t_empty[2];
  uint32_t tmem;
  uint32_t stop;
};

// What every role derives alike for a unit.
struct Unit {
  int b, t0, tokens, tile0, tile1;
};

__device__ __forceinline__ int length_of(const ScoreParams& p, int b, int t) {
  const int n = p.a.lengths[static_cast<int64_t>(b) * p.a.T + t];
  return n < 0 ? 0 : min(static_cast<int64_t>(n), p.a.width);
}

__device__ __forceinline__ Unit unit_of(const ScoreParams& p, int64_t u) {
  Unit r;
  const int64_t c = u / p.groups;
  r.t0 = static_cast<int>(u - c * p.groups) * p.tokens;
  r.b = static_cast<int>(c / p.chunks);
  r.tokens = min(p.tokens, p.a.T - r.t0);
  const int lane = threadIdx.x & 31;
  const int longest = __reduce_max_sync(0xffffffffu, lane < r.tokens ? length_of(p, r.b, r.t0 + lane) : 0);
  r.tile0 = static_cast<int>(c - static_cast<int64_t>(r.b) * p.chunks) * p.unit_tiles;
  r.tile1 = min(r.tile0 + p.unit_tiles, longest / kTile + (longest % kTile != 0));
  return r;
}

__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
// max(0, x), a NaN kept, of two products.
__device__ __forceinline__ uint64_t relu2(uint32_t x, uint32_t y) {
  uint64_t r;
  asm("{\n\t.reg .f32 a, b;\n\tmax.NaN.f32 a, %1, 0f00000000;\n\tmax.NaN.f32 b, %2, 0f00000000;\n\t"
      "mov.b64 %0, {a, b};\n\t}"
      : "=l"(r)
      : "f"(__uint_as_float(x)), "f"(__uint_as_float(y)));
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

// Queries, weights and lengths of a unit into buffer `buf`, by `n` threads.
template <typename E>
__device__ __forceinline__ void fetch_queries(const ScoreParams& p, const Unit& r, unsigned char* smem, uint32_t q_bytes,
                                              ScoreShared& sh, uint32_t buf, int th, int n, const void* nowhere) {
  const E* q = static_cast<const E*>(p.a.q) + r.b * p.a.q_seq_stride;
  const int units = p.blocks * 8;
  for (int i = th; i < p.cols * units; i += n) {
    const int col = i / units, j = i - col * units;
    const int t = col / p.hp, h = col - t * p.hp;
    const bool real = t < r.tokens && h < p.a.H && j < p.row_units;
    const E* src = real ? q + (r.t0 + t) * p.a.q_token_stride + h * p.a.q_head_stride + j * (16 / sizeof(E)) : nullptr;
    const uint32_t at = buf * q_bytes + (j >> 3) * p.cols * 128 + swizzled(col, j & 7);
    if (p.q_vector) {
      copy16(smem_addr(smem) + at, real ? src : nowhere, real);
    } else {
      E v[16 / sizeof(E)];
      for (int e = 0; e < static_cast<int>(16 / sizeof(E)); ++e) v[e] = real ? src[e] : E(0.0f);
      *reinterpret_cast<uint4*>(smem + at) = *reinterpret_cast<const uint4*>(v);
    }
  }
  for (int i = th; i < p.cols; i += n) {
    const int t = i / p.hp, h = i - t * p.hp;
    sh.weights[buf][i] =
        t < r.tokens && h < p.a.H ? p.a.weights[(static_cast<int64_t>(r.b) * p.a.T + r.t0 + t) * p.a.H + h] : 0.0f;
  }
  if (th < kMaxTokens) sh.lengths[buf][th] = th < r.tokens ? length_of(p, r.b, r.t0 + th) : 0;
  copy_arrive(&sh.q_full[buf]);
  mbar_arrive(&sh.q_full[buf]);
}

// STAGES tiles of keys in flight; STEP columns per TMEM load; keys by BOXES of
// the TMA engine or by 16-byte copies.
template <typename E, int STAGES, int STEP, bool BOXES>
__global__ void __launch_bounds__(kScoreThreads, 1) scores_kernel(const __grid_constant__ ScoreParams p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t q_bytes = static_cast<uint32_t>(p.cols) * 128 * p.blocks;
  const uint32_t tile_bytes = kTile * 128 * p.blocks;
  unsigned char* ring = smem + 2 * q_bytes;
  ScoreShared& sh = *reinterpret_cast<ScoreShared*>(ring + STAGES * tile_bytes);
  const uint32_t q_addr = smem_addr(smem), ring_addr = smem_addr(ring);

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&sh.full[i], BOXES ? 1 : 128), mbar_init(&sh.empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], BOXES ? 192 : 256);  // the copies' arrivals and the stores'
      mbar_init(&sh.q_empty[i], 1 + kEpilogueWarps);
      mbar_init(&sh.t_full[i], 1);
      mbar_init(&sh.t_empty[i], 128);
    }
    sh.stop = 0;
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile uint32_t* stop = &sh.stop;

  // what a copy of nothing points at
  const void* nowhere = reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(p.a.q) & ~static_cast<uintptr_t>(15));
  if (BOXES && warp == 8) {
    // ---- keys, by boxes: lane i fetches block i / 16 of the box i % 16 of a tile ----
    const int box = lane & 15, block = lane >> 4, boxes = kTile / p.box_rows;
    const bool mine = box < boxes && block < p.blocks;
    uint32_t k = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
      const Unit r = unit_of(p, u);
      if (r.tile0 >= r.tile1) continue;
      const int32_t* table = p.a.page_table + r.b * p.a.table_stride;
      auto entry = [&](int tile) -> int64_t { return static_cast<int64_t>(tile) * kTile + box * p.box_rows; };
      auto page_at = [&](int tile) -> int32_t {
        const int64_t s = entry(tile);
        return mine && tile < r.tile1 && s < p.a.width ? table[static_cast<int32_t>(s) / p.a.page_size] : -1;
      };
      int32_t next = page_at(r.tile0);  // read a tile ahead
      for (int tile = r.tile0; tile < r.tile1; ++tile, ++k) {
        const uint32_t stage = k % STAGES;
        const int32_t page = next;
        next = page_at(tile + 1);
        ok = wait_or_stop(&sh.empty[stage], ((k / STAGES) & 1) ^ 1, stop);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[stage], tile_bytes);
        __syncwarp();
        if (mine) {
          const int z = page < 0 || page >= p.a.num_pages ? static_cast<int>(p.a.num_pages) : page;  // absent: zeros
          const int y = static_cast<int>(static_cast<uint32_t>(entry(tile)) % static_cast<uint32_t>(p.a.page_size));
          box_load(ring_addr + stage * tile_bytes + (block * kTile + box * p.box_rows) * 128, &p.map,
                   block * (128 / static_cast<int>(sizeof(E))), y, z, &sh.full[stage]);
        }
      }
    }
    // no box may arrive after the CTA has left
    for (uint32_t i = 0; i < STAGES && i < k; ++i)
      mbar_wait_bounded(&sh.full[(k - 1 - i) % STAGES], ((k - 1 - i) / STAGES) & 1, 1000000000ull);
  } else if (BOXES && warp > 8 && warp < 12) {
    // ---- queries, a unit ahead ----
    uint32_t nu = 0;
    for (int64_t u = blockIdx.x; u < p.units; u += gridDim.x) {
      const Unit r = unit_of(p, u);
      if (r.tile0 >= r.tile1) continue;
      if (!wait_or_stop(&sh.q_empty[nu & 1], ((nu >> 1) & 1) ^ 1, stop)) break;
      fetch_queries<E>(p, r, smem, q_bytes, sh, nu & 1, threadIdx.x - 288, 96, nowhere);
      ++nu;
    }
    copy_commit();
    copy_wait<0>();
  } else if (!BOXES && warp >= 8 && warp < 12) {
    // ---- keys and queries, by 16-byte copies: 8 lanes fetch a row's 128 bytes ----
    const int w = warp - 8;
    const uint32_t unit16 = lane & 7;
    uint32_t k = 0, nu = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
      const Unit r = unit_of(p, u);
      if (r.tile0 >= r.tile1) continue;
      const int32_t* table = p.a.page_table + r.b * p.a.table_stride;
      // this lane looks up row 32 w + lane of a tile
      auto entry = [&](int tile) -> int64_t { return static_cast<int64_t>(tile) * kTile + w * 32 + lane; };
      auto page_at = [&](int tile) -> int32_t {
        const int64_t s = entry(tile);
        return tile < r.tile1 && s < p.a.width ? table[static_cast<int32_t>(s) / p.a.page_size] : -1;
      };
      int32_t next = page_at(r.tile0);  // read a tile ahead
      ok = wait_or_stop(&sh.q_empty[nu & 1], ((nu >> 1) & 1) ^ 1, stop);
      if (!ok) break;
      fetch_queries<E>(p, r, smem, q_bytes, sh, nu & 1, threadIdx.x - 256, 128, nowhere);
      ++nu;
      for (int tile = r.tile0; tile < r.tile1; ++tile, ++k) {
        const uint32_t stage = k % STAGES;
        const int32_t page = next;
        next = page_at(tile + 1);
        ok = wait_or_stop(&sh.empty[stage], ((k / STAGES) & 1) ^ 1, stop);
        if (!ok) break;
        const int64_t slot = page < 0 || page >= p.a.num_pages
                                 ? -1
                                 : page * p.a.key_page_stride +
                                       static_cast<int32_t>(entry(tile)) % p.a.page_size * p.a.key_token_stride;
        const uint32_t dst = ring_addr + stage * tile_bytes;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = 4 * i + (lane >> 3);
          const int64_t s = __shfl_sync(0xffffffffu, slot, row);
          const E* src = static_cast<const E*>(p.a.keys) + (s < 0 ? 0 : s);
          for (int c = 0; c < p.blocks; ++c) {
            const uint32_t j = c * 8 + unit16;
            const bool real = s >= 0 && j < static_cast<uint32_t>(p.row_units);
            copy16(dst + c * kTile * 128 + swizzled(w * 32 + row, unit16), real ? src + j * (16 / sizeof(E)) : nowhere,
                   real);
          }
        }
        copy_arrive(&sh.full[stage]);
      }
    }
    copy_commit();
    copy_wait<0>();
  } else if (warp == 12) {
    // ---- products ----
    const uint32_t desc = mma_desc(Kind<E>::type, p.cols);
    uint32_t k = 0, nu = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
      const Unit r = unit_of(p, u);
      if (r.tile0 >= r.tile1) continue;
      const uint32_t buf = nu & 1;
      ok = wait_or_stop(&sh.q_full[buf], (nu >> 1) & 1, stop);
      ++nu;
      for (int tile = r.tile0; tile < r.tile1 && ok; ++tile, ++k) {
        const uint32_t stage = k % STAGES, tb = k & 1;
        ok = wait_or_stop(&sh.t_empty[tb], ((k >> 1) & 1) ^ 1, stop) &&
             wait_or_stop(&sh.full[stage], (k / STAGES) & 1, stop);
        if (!ok) break;
        fence_proxy_async_smem();  // the 16-byte copies are in; now the tensor cores may see them
        tc_fence_after();
        if (lane == 0) {
          for (int c = 0; c < p.blocks; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint64_t da = operand_desc(ring_addr + stage * tile_bytes + c * kTile * 128 + j * 32);
              const uint64_t db = operand_desc(q_addr + buf * q_bytes + c * p.cols * 128 + j * 32);
              if constexpr (sizeof(E) == 1)
                mma_f8(tmem + tb * kMaxCols, da, db, desc, c + j > 0);
              else
                mma_f16(tmem + tb * kMaxCols, da, db, desc, c + j > 0);
            }
          mma_commit(&sh.empty[stage]);
          mma_commit(&sh.t_full[tb]);
          if (tile + 1 == r.tile1) mma_commit(&sh.q_empty[buf]);
        }
        __syncwarp();
      }
    }
    // every product is complete before the memory it uses goes away
    for (uint32_t i = 0; i < 2 && i < k; ++i)
      wait_or_stop(&sh.t_full[(k - 1 - i) & 1], ((k - 1 - i) >> 1) & 1, stop);
  } else {
    // ---- sums over heads ----
    const int group = warp >> 2, quarter = warp & 3;
    uint32_t k = 0, nu = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
      const Unit r = unit_of(p, u);
      if (r.tile0 >= r.tile1) continue;
      const uint32_t buf = nu & 1;
      ok = wait_or_stop(&sh.q_full[buf], (nu >> 1) & 1, stop);
      if (!ok) break;
      ++nu;
      float* out = p.a.out + r.b * p.a.out_seq_stride + r.t0 * p.a.out_token_stride;
      const int32_t* table = p.a.page_table + r.b * p.a.table_stride;
      auto entry = [&](int tile) -> int64_t { return static_cast<int64_t>(tile) * kTile + quarter * 32 + lane; };
      auto page_at = [&](int tile) -> int32_t {
        const int64_t s = entry(tile);
        return tile < r.tile1 && s < p.a.width ? table[static_cast<int32_t>(s) / p.a.page_size] : -1;
      };
      const int mine = r.tile0 + static_cast<int>((k ^ group) & 1);  // this group's tiles: every other one
      int32_t next = page_at(mine);
      const uint32_t k0 = k;
      k += mine - r.tile0;
      for (int tile = mine; tile < r.tile1; tile += 2, k += 2) {
        const int64_t s = entry(tile);
        const int32_t page = next;
        next = page_at(tile + 2);
        const bool absent = page < 0 || page >= p.a.num_pages;
        float scale = 1.0f;
        if (!absent && p.a.key_scales != nullptr)
          scale = p.a.key_scales[static_cast<int64_t>(page) * p.a.page_size + static_cast<int32_t>(s) % p.a.page_size];
        ok = wait_or_stop(&sh.t_full[group], (k >> 1) & 1, stop);
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = tmem + group * kMaxCols + (static_cast<uint32_t>(quarter) << 21);
        for (int t = 0; t < r.tokens; ++t) {
          uint64_t acc[4] = {};
          const float* wt = sh.weights[buf] + t * p.hp;
          for (int c = 0; c < p.hp; c += STEP) {
            uint32_t v[STEP];
            tmem_ld(v, at + t * p.hp + c);
            tmem_wait_ld(v);
#pragma unroll
            for (int j = 0; j < STEP; j += 4) {
              const ulonglong2 ww = *reinterpret_cast<const ulonglong2*>(wt + c + j);
              fma2(acc[(j / 2) & 3], relu2(v[j], v[j + 1]), ww.x);
              fma2(acc[(j / 2 + 1) & 3], relu2(v[j + 2], v[j + 3]), ww.y);
            }
          }
          float sum = 0.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            sum += __uint_as_float(static_cast<uint32_t>(acc[j])) + __uint_as_float(static_cast<uint32_t>(acc[j] >> 32));
          if (t == r.tokens - 1) {  // the buffer is read: the next product may have it
            tc_fence_before();
            mbar_arrive(&sh.t_empty[group]);
          }
          if (s < sh.lengths[buf][t])
            out[t * p.a.out_token_stride + s] = absent ? __int_as_float(0xff800000) : sum * scale;
        }
      }
      k = k0 + (r.tile1 - r.tile0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_empty[buf]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*stop != 0) {  // a wait ran out: NaN, not half a result
    for (int64_t u = blockIdx.x; u < p.units; u += gridDim.x) {
      const Unit r = unit_of(p, u);
      for (int t = 0; t < r.tokens; ++t) {
        const int64_t end = min(static_cast<int64_t>(r.tile1) * kTile, static_cast<int64_t>(length_of(p, r.b, r.t0 + t)));
        for (int64_t s = static_cast<int64_t>(r.tile0) * kTile + threadIdx.x; s < end; s += kScoreThreads)
          p.a.out[r.b * p.a.out_seq_stride + (r.t0 + t) * p.a.out_token_stride + s] = __int_as_float(0x7fc00000);
      }
    }
  }
  if (warp == 12) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

template <typename E, int STAGES, int STEP, bool BOXES>
topk_status launch_variant(const ScoreParams& p, int dev, int sm_count, cudaStream_t stream) {
  static_assert(sizeof(ScoreShared) <= 3072, "barriers and weights");
  const size_t bytes = 2 * static_cast<size_t>(p.cols) * 128 * p.blocks + STAGES * static_cast<size_t>(kTile) * 128 * p.blocks +
                       sizeof(ScoreShared);
  constexpr auto kernel = scores_kernel<E, STAGES, STEP, BOXES>;
  const topk_status st = allow_shared<kernel>(dev);
  if (st != TOPK_OK) return st;
  const int64_t grid = p.units < sm_count ? p.units : sm_count;
  kernel<<<static_cast<unsigned>(grid), kScoreThreads, bytes, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? TOPK_OK : TOPK_ECUDA;
}

template <typename E, int STAGES, int STEP>
topk_status launch_step(const ScoreParams& p, int dev, int sm_count, cudaStream_t stream) {
  return p.box_rows > 0 ? launch_variant<E, STAGES, STEP, true>(p, dev, sm_count, stream)
                        : launch_variant<E, STAGES, STEP, false>(p, dev, sm_count, stream);
}

template <typename E, int STEP>
topk_status launch_ring(const ScoreParams& p, int dev, int sm_count, cudaStream_t stream) {
  // The ring gets what the queries leave of 227 KB: 6, 5 or 3 tiles.
  if (p.cols <= 64) return launch_step<E, 6, STEP>(p, dev, sm_count, stream);
  if (p.cols <= 128) return launch_step<E, 5, STEP>(p, dev, sm_count, stream);
  return launch_step<E, 3, STEP>(p, dev, sm_count, stream);
}

template <typename E>
topk_status launch_typed(const sparse_scores_args& a, int dev, int sm_count, cudaStream_t stream) {
  ScoreParams p = {};
  p.a = a;
  const int size = sizeof(E);
  p.hp = (a.H + 15) / 16 * 16;
  p.tokens = kMaxCols / p.hp < kMaxTokens ? kMaxCols / p.hp : kMaxTokens;
  if (p.tokens > a.T) p.tokens = a.T;
  p.cols = p.tokens * p.hp;
  p.blocks = (a.D * size + 127) / 128;
  p.row_units = a.D * size / 16;
  p.groups = (a.T + p.tokens - 1) / p.tokens;
  // Work units of at most 16 tiles: enough of them to even out the SMs, long
  // enough to hide the next unit's queries; fewer tiles while SMs would idle.
  const int64_t tiles = (a.width + kTile - 1) / kTile;
  const int64_t all = tiles * a.B * p.groups;
  int64_t per = (all + sm_count - 1) / sm_count;
  p.unit_tiles = static_cast<int32_t>(per < 16 ? per : 16);
  p.chunks = static_cast<int32_t>((tiles + p.unit_tiles - 1) / p.unit_tiles);
  p.units = static_cast<int64_t>(p.chunks) * p.groups * a.B;
  p.q_vector = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && a.q_seq_stride * size % 16 == 0 &&
               a.q_token_stride * size % 16 == 0 && a.q_head_stride * size % 16 == 0;
  // Boxes hold entries of one page: the largest power of two that divides the
  // page, where it is at least 8, the rows of a swizzle group.
  int rows = a.page_size & -a.page_size;
  rows = rows < kTile ? rows : kTile;
  const bool boxes = rows >= 8 && paged_map(&p.map, Kind<E>::map_type, size, a.keys, a.D, a.page_size, a.num_pages,
                                            a.key_token_stride, a.key_page_stride, rows);
  p.box_rows = boxes ? rows : 0;
  return p.hp % 32 == 0 ? launch_ring<E, 32>(p, dev, sm_count, stream) : launch_ring<E, 16>(p, dev, sm_count, stream);
}

}  // namespace

topk_status launch_scores(const sparse_scores_args& a, int dev, int sm_count, cudaStream_t stream) {
  switch (a.type) {
    case SPARSE_BF16: return launch_typed<__nv_bfloat16>(a, dev, sm_count, stream);
    case SPARSE_FP16: return launch_typed<__half>(a, dev, sm_count, stream);
    default: return launch_typed<__nv_fp8_e4m3>(a, dev, sm_count, stream);
  }
}

}  // namespace tki
