// Attention over the selected entries of a paged cache
// (include/sparse_step.h, sparse_attention).
//
// One pass over the selected entries, 64 at a time, with the running maximum
// and sum of a softmax: S = Q K^T and O += P V on the tensor cores, with the
// query heads that share a key head as the 128 rows (TMEM lanes) of both, S, P
// and O in TMEM, and one thread per row between them.
//
// Rows. Groups of up to 32 (64) heads leave 128 rows mostly empty, so they
// are laid out in 4 (2) copies, and copy i of a row takes every tile's i-th
// part of 64 / copies entries, with zero weights elsewhere: the copies' warps
// share the exponentials, and their sums are joined at the end like those of
// CTAs that share a row. The products cost the same either way.
//
// Rescaling. Each row keeps a reference r for its weights 2^(z - r) and moves
// it only when the maximum has grown past r + 8, so that O in TMEM is rarely
// touched; weights are then at most 2^8, which both types hold.
//
// Few rows. The tiles of a row are dealt over a cluster of up to 8 CTAs,
// which join their sums through distributed shared memory: one launch, no
// workspace, the same order on every call.
//
// Warps 0-3: softmax, one row per thread; 4-11: gather entries through the page
// table with 16-byte asynchronous copies, zeros for what is not seen, in two
// sets that take tiles in turn; 12 and 13: one thread each issues Q K^T and
// P V. Keys and values have rings of their own, filled by two warps of a set
// each: a stage of keys is free again right after Q K^T, so the gathers run
// ahead of the softmax (one ring of both, two stages deep, left every tile
// waiting for its gather).
//
// Precision. Scores, statistics and O are FP32; a weight 2^(z - r) is rounded
// once to the type of v, the operand type of the second product, half a step
// (2^-8 in bf16) relative to itself; the sum that divides adds the unrounded ones.
//
// Measured: 64 rows x 2048 entries x 8 key heads of 128, bf16, capped, 92 us,
// 5.9 TB/s of random 256-byte reads (79 us for its bytes at the measured copy
// rate). 2048 rows x 512 entries of 256 + 192 shared, 64 heads: 131 us, the tensor
// pipe busy in 40 % of the cycles (31 us at the measured matrix rate). Four rows x
// 512 entries: 8.5 us, two tiles a CTA and one exchange.
#include <cuda_runtime.h>

#include <cstdint>

#include "attention_math.cuh"
#include "step_launch.cuh"
#include "tcgen05.cuh"

namespace tki {
namespace {

constexpr int kKeys = 64;  // entries per tile
constexpr int kGatherWarps = 8, kMmaWarp = 4 + kGatherWarps;
constexpr int kAttThreads = (kMmaWarp + 2) * 32;  // Q K^T, then P V
constexpr int kMaxStages = 6;
// Masks outlive their keys' stage: tile j's are written when the products of
// tile j - stages are issued, which follow the softmax of the tile kMaxBufs
// before at the latest.
constexpr int kMaxBufs = 3;  // buffers of scores and weights in TMEM
constexpr int kMasks = kMaxStages + kMaxBufs;
constexpr float kGrowth = 8.0f;

struct AttParams {
  sparse_attention_args a;
  int32_t heads;      // query heads per key head
  int32_t m_tiles;    // tiles of 128 rows per key head
  uint32_t works;     // (row, key head, tile of rows)
  int32_t d_blocks, v_blocks;  // 128-byte blocks of an entry's keys and values
  int32_t shared;     // v is a prefix of k's entries
  int32_t page_shift;  // log2 of page_size, or -1
  uint32_t pages, table_width;
  int32_t k_stages, v_stages;  // of the rings; no second ring when shared
  int32_t k_bytes, v_bytes;    // of a stage
  int32_t k_at, v_at;          // the rings, after Q
  int32_t shared_at, parts_at;  // AttShared, AttParts
  int32_t tmem_cols, bufs;
  float scale_log2e;                // of a product, to a logit in units of log 2
  float scale_over_cap, cap_log2e;  // with a cap
  bool q_vector;
};

struct AttShared {
  float away[kMasks][kKeys];           // position - query's, per entry of a tile
  uint32_t seen[kMasks][2];            // bit per entry
  float top[128], sum[128];            // of the rows
  float head_top[128], head_sum[128];  // of the heads, the copies joined; 1 / sum in a CTA that is alone
  uint64_t k_full[kMaxStages], v_full[kMaxStages], masks[kMasks], q_full;
  // Of tile i at i % 8: scores there, weights there, products with v done.
  // Nobody who waits on one lags behind by eight tiles.
  uint64_t s_full[8], p_full[8], pv_done[8];
  uint64_t q_empty, o_free;  // Q used up, O read: between one work and the next
  uint64_t drained[2];       // of the threads that issue Q K^T and P V
  uint32_t tmem;
  uint32_t stop;
};

// With two copies of the heads: 32 columns of rows on their way from one copy
// to the other, padded.
struct AttParts {
  float part[2][64][36];
};

__host__ __device__ __forceinline__ int tiles_of(int32_t entries) { return entries / kKeys + (entries % kKeys != 0); }

struct Work {
  int g, heads, head0;  // key head; real rows, and the first one's query head
  int64_t row, b, t;
};

__device__ __forceinline__ Work work_of(const AttParams& p, uint32_t w) {
  Work r;
  const uint32_t pair = w / static_cast<uint32_t>(p.m_tiles), row = pair / static_cast<uint32_t>(p.a.Hkv);
  const int m_tile = static_cast<int>(w - pair * p.m_tiles);
  const uint32_t b = row / static_cast<uint32_t>(p.a.T);
  r.g = static_cast<int>(pair - row * p.a.Hkv);
  r.heads = min(p.heads - m_tile * 128, 128);
  r.head0 = r.g * p.heads + m_tile * 128;
  r.row = row, r.b = b, r.t = row - b * static_cast<uint32_t>(p.a.T);
  return r;
}

// The four softmax warps among themselves.
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Q of a work, by 128 threads, 8 per 128 bytes of a row; each arrives twice.
template <typename E, int COPIES>
__device__ __forceinline__ void fetch_queries(const AttParams& p, const Work& k, unsigned char* smem, uint64_t* q_full, int th) {
  const sparse_attention_args& a = p.a;
  const void* nowhere = reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(a.q) & ~static_cast<uintptr_t>(15));
  const int unit16 = th & 7, sub = th >> 3;
  const E* q = static_cast<const E*>(a.q) + k.b * a.q_seq_stride + k.t * a.q_token_stride + k.head0 * a.q_head_stride;
  for (int c = 0; c < p.d_blocks; ++c) {
    const int d = c * 64 + unit16 * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = 16 * j + sub, h = r % (128 / COPIES);
      const bool real = h < k.heads && d < a.D;
      const uint32_t at = c * (128 * 128) + swizzled(r, unit16);
      const E* src = q + h * a.q_head_stride + d;
      if (p.q_vector) {
        copy16(smem_addr(smem) + at, real ? src : nowhere, real);
      } else {
        alignas(16) E v[8];
        for (int e = 0; e < 8; ++e) v[e] = real ? src[e] : E(0.0f);
        *reinterpret_cast<uint4*>(smem + at) = *reinterpret_cast<const uint4*>(v);
      }
    }
  }
  copy_arrive(q_full);
  mbar_arrive(q_full);
}

// A row's factor, 1 / its sum of weights: zero where nothing is seen.
__device__ __forceinline__ float inverse(float all, float total) {
  return total != total ? total : is_low(all) ? 0.0f : 1.0f / total;
}
__device__ __forceinline__ float logsum(float all, float total) {
  return total != total ? total : is_low(all) ? all : (all + log2f(total)) * kLn2;
}

template <typename E, int COPIES>
__global__ void __launch_bounds__(kAttThreads, COPIES == 4 ? 2 : 1)
    attention_kernel(const __grid_constant__ AttParams p, const int cluster) {
  extern __shared__ __align__(1024) unsigned char smem[];
  constexpr int kPart = kKeys / COPIES;             // entries of a tile that a row's copy takes
  constexpr int kStep = kPart < 32 ? kPart : 32;    // columns per TMEM load
  constexpr int kRows = 128 / COPIES;               // rows of one copy
  AttShared& sh = *reinterpret_cast<AttShared*>(smem + p.shared_at);
  const sparse_attention_args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster > 1 ? cluster_ctarank() : 0;
  // With one or two copies a CTA stays for several works, its roles running
  // into the next one while the softmax warps end the last.
  constexpr bool kStay = COPIES <= 2;
  const uint32_t step_w = gridDim.x / cluster;
  Work k = work_of(p, blockIdx.x / cluster);
  const int all_tiles = tiles_of(a.K);
  const int tiles = all_tiles > static_cast<int>(rank) ? (all_tiles - static_cast<int>(rank) + cluster - 1) / cluster : 0;
  const uint32_t base = smem_addr(smem);
  const uint32_t k_ring = base + p.k_at, v_ring = base + p.v_at;

  const int half = warp & 1;  // of a tile's entries
  const int32_t* indices = nullptr;
  const int32_t* table = nullptr;
  int32_t last = INT32_MAX, first = 0;
  auto look_at = [&](const Work& k) {
    indices = a.indices + k.row * a.K;
    table = a.page_table != nullptr ? a.page_table + k.b * a.table_stride : nullptr;
    last = a.query_positions != nullptr ? a.query_positions[k.row] : INT32_MAX;
    first = a.first != nullptr ? max(a.first[k.row], 0) : 0;
  };
  const bool some = a.page_size > 0 && a.num_pages > 0;
  // Gathering: each lane looks up one entry of a tile, its index two of
  // the warp's tiles ahead, its page id one.
  auto index_of = [&](int i) -> int32_t {
    const int64_t j = (static_cast<int64_t>(i) * cluster + rank) * kKeys + half * 32 + lane;
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
  const bool gathers = warp >= 4 && warp < kMmaWarp;
  const int turn = (warp - 4) >> 2;  // of the two sets of gathering warps, which take tiles in turn
  if (gathers) look_at(k);
  int32_t pos = gathers ? index_of(turn) : -1, pos1 = gathers ? index_of(turn + 2) : -1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.k_stages; ++i) mbar_init(&sh.k_full[i], p.shared ? 128 : 64);
    for (int i = 0; i < p.v_stages; ++i) mbar_init(&sh.v_full[i], 64);
    for (int i = 0; i < kMasks; ++i) mbar_init(&sh.masks[i], 2);
    mbar_init(&sh.q_full, 256);
    for (int i = 0; i < 8; ++i) mbar_init(&sh.s_full[i], 1), mbar_init(&sh.p_full[i], 128), mbar_init(&sh.pv_done[i], 1);
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.o_free, 128);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.drained[i], 1);
    sh.stop = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&sh.tmem, p.tmem_cols);
  uint32_t page = page_of(pos);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem, tmem_o = tmem + p.bufs * kKeys;
  volatile uint32_t* stop = &sh.stop;
  bool one = false;  // a thread that issues products

  float top = __int_as_float(0xff800000), sum = 0.0f;  // of this thread's row (its reference and sum of weights)

  if (gathers) {
    // ---- gather ----
    // Warps 0 and 1 fetch the tile's entries 0-31 and 32-63, keys; warps 2
    // and 3 their values, or the second half of their blocks when shared.
    const int w = (warp - 4) & 3;
    const bool values = w >= 2 && !p.shared;
    const int split = (p.d_blocks + 1) / 2;  // shared: blocks of the first two warps
    const int c0 = w >= 2 && p.shared ? split : 0;
    const int c1 = values ? p.v_blocks : w < 2 && p.shared ? split : p.d_blocks;
    const int dim = values ? a.Dv : a.D;
    const int64_t head_stride = values ? a.v_head_stride : a.k_head_stride;
    const int64_t page_stride = values ? a.v_page_stride : a.k_page_stride;
    const int64_t token_stride = values ? a.v_token_stride : a.k_token_stride;
    uint64_t* full = values ? sh.v_full : sh.k_full;
    uint64_t* used = values || p.shared ? sh.pv_done : sh.s_full;  // when a tile's stage is free
    const int stages = values ? p.v_stages : p.k_stages, stage_bytes = values ? p.v_bytes : p.k_bytes;
    // 8 lanes fetch 128 bytes of an entry; step j has entries 4 j + lane / 8.
    const uint32_t unit16 = lane & 7, sub = lane >> 3;
    const uint32_t at = (values ? v_ring : k_ring) + (half * 32 + sub) * 128;
    const uint32_t even = (unit16 ^ sub) << 4, odd = (unit16 ^ (sub + 4)) << 4;
    bool ok = true;
    int n = 0, stage = turn;  // tiles before this work; n + i is a tile's number in the CTA
    for (uint32_t w_at = blockIdx.x / cluster, nw = 0; w_at < p.works && ok; w_at += step_w, ++nw, n += tiles) {
    const int i0 = (turn - n) & 1;  // the set's tiles: every other number
    if (nw > 0) {
      k = work_of(p, w_at);
      look_at(k);
      pos = index_of(i0), pos1 = index_of(i0 + 2);
      if (tiles > 0 && turn == 0) {
        ok = wait_or_stop(&sh.q_empty, (nw - 1) & 1, stop);
        if (!ok) break;
        fetch_queries<E, COPIES>(p, k, smem, &sh.q_full, threadIdx.x - 128);
      }
      page = page_of(pos);
    }
    // an empty cache has no address: nothing is read from the one it gets
    const E* mine = some ? static_cast<const E*>(values ? a.v : a.k) + k.g * head_stride + unit16 * 8
                         : reinterpret_cast<const E*>(reinterpret_cast<uintptr_t>(a.q) & ~static_cast<uintptr_t>(15));
    for (int i = i0; i < tiles; i += 2) {
      const int32_t pos2 = index_of(i + 4);
      const uint32_t page1 = page_of(pos1);
      const bool seen = page < p.pages;
      const uint32_t place = static_cast<uint32_t>(pos) - page_index(pos) * static_cast<uint32_t>(a.page_size);
      const int64_t entry = seen ? page * page_stride + place * token_stride : 0;
      const uint32_t bits = __ballot_sync(0xffffffffu, seen);
      const int before = n + i - stages;
      ok = before < 0 || wait_or_stop(&used[before & 7], (before >> 3) & 1, stop);
      if (!ok) break;
      const uint32_t dst = at + stage * stage_bytes;
      const E* from[8];
      uint32_t bytes[8];  // to copy: none of an entry that is not seen, whose place stays zero
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        from[j] = mine + __shfl_sync(0xffffffffu, entry, 4 * j + sub);
        bytes[j] = (bits >> (4 * j + sub)) & 1 ? 16 : 0;
      }
#pragma unroll
      for (int c = 0; c < SPARSE_ATTENTION_MAX_D / 64; ++c) {
        if (c < c0 || c >= c1) continue;
        if (c * 64 + 64 <= dim) {
#pragma unroll
          for (int j = 0; j < 8; ++j) copy_bytes(dst + c * (kKeys * 128) + j * 512 + (j & 1 ? odd : even), from[j] + c * 64, bytes[j]);
        } else {  // the last block of a dimension that does not fill it
          const bool inside = c * 64 + static_cast<int>(unit16) * 8 < dim;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            copy_bytes(dst + c * (kKeys * 128) + j * 512 + (j & 1 ? odd : even), inside ? from[j] + c * 64 : mine,
                       inside ? bytes[j] : 0);
        }
      }
      copy_arrive(&full[stage]);
      if (w < 2) {
        const int mask = (n + i) % kMasks;
        sh.away[mask][half * 32 + lane] = static_cast<float>(seen ? pos - last : 0);
        if (lane == 0) sh.seen[mask][half] = bits;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.masks[mask]);
      }
      pos = pos1, pos1 = pos2, page = page1;
      stage += 2;
      if (stage >= stages) stage -= stages;
    }
    if (!kStay) break;
    }
    copy_commit();
    copy_wait<0>();
  } else if (warp == kMmaWarp) {
    // ---- S = Q K^T, by one thread, whose waits need no vote ----
    one = elect_one();
    if (tiles > 0 && one) {
      const uint32_t desc = mma_desc(Pack<E>::type, kKeys);
      const uint64_t q_desc = operand_desc(base), k_desc = operand_desc(k_ring);
      int stage = 0, turn_of = 0, n = 0;
      uint32_t to = tmem;
      bool ok = true;
      for (uint32_t w_at = blockIdx.x / cluster, nw = 0; w_at < p.works && ok; w_at += step_w, ++nw) {
        ok = wait_or_stop_one(&sh.q_full, nw & 1, stop);
        for (int i = 0; i < tiles && ok; ++i, ++n) {
          const int before = n - p.bufs;  // these scores go where its weights were
          ok = (before < 0 || wait_or_stop_one(&sh.pv_done[before & 7], (before >> 3) & 1, stop)) &&
               wait_or_stop_one(&sh.k_full[stage], turn_of, stop);
          if (!ok) break;
          fence_proxy_async_smem();
          tc_fence_after();
          const uint64_t kd = k_desc + static_cast<uint32_t>(stage * p.k_bytes >> 4);
          for (int c = 0; c < p.d_blocks; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_f16(to, q_desc + static_cast<uint32_t>(c * (128 * 128 >> 4) + j * 2),
                      kd + static_cast<uint32_t>(c * (kKeys * 128 >> 4) + j * 2), desc, c + j > 0);
          mma_commit(&sh.s_full[n & 7]);
          if (++stage == p.k_stages) stage = 0, turn_of ^= 1;
          to = to + kKeys == tmem_o ? tmem : to + kKeys;
        }
        if (ok) mma_commit(&sh.q_empty);
        if (!kStay) break;
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp + 1) {
    // ---- O += P V, by another, so that neither's waits hold up the other ----
    one = elect_one();
    if (tiles > 0 && one) {
      const uint32_t desc = mma_desc(Pack<E>::type, (a.Dv + 15) / 16 * 16, true);
      const uint64_t v_desc = operand_desc(p.shared ? k_ring : v_ring, kKeys * 128);
      const int stages = p.shared ? p.k_stages : p.v_stages, stage_bytes = p.shared ? p.k_bytes : p.v_bytes;
      uint64_t* full = p.shared ? sh.k_full : sh.v_full;
      int stage = 0, turn_of = 0, n = 0;
      uint32_t from = tmem;
      bool ok = true;
      for (uint32_t w_at = blockIdx.x / cluster, nw = 0; w_at < p.works && ok; w_at += step_w, ++nw) {
        if (nw > 0) ok = wait_or_stop_one(&sh.o_free, (nw - 1) & 1, stop);
        for (int i = 0; i < tiles && ok; ++i, ++n) {
          ok = wait_or_stop_one(&full[stage], turn_of, stop);
          fence_proxy_async_smem();
          ok = ok && wait_or_stop_one(&sh.p_full[n & 7], (n >> 3) & 1, stop);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = v_desc + static_cast<uint32_t>(stage * stage_bytes >> 4);
#pragma unroll
          for (int j = 0; j < kKeys / 16; ++j)
            mma_f16_ts(tmem_o, from + j * 8, vd + static_cast<uint32_t>(j * (16 * 128 >> 4)), desc, i + j > 0);
          mma_commit(&sh.pv_done[n & 7]);
          if (++stage == stages) stage = 0, turn_of ^= 1;
          from = from + kKeys == tmem_o ? tmem : from + kKeys;
        }
        if (!kStay) break;
      }
    }
    __syncwarp();
  } else {
    // ---- softmax ----
    const int copy = threadIdx.x / kRows;
    if (tiles > 0) fetch_queries<E, COPIES>(p, k, smem, &sh.q_full, threadIdx.x);  // the first work's
    const int h = threadIdx.x % kRows;
    const float scale = p.scale_log2e;
    const uint32_t lanes = static_cast<uint32_t>(warp) << 21;
    uint32_t buf = 0;
    int n = 0;  // tiles before this work
    for (uint32_t w_at = blockIdx.x / cluster, nw = 0; w_at < p.works; w_at += step_w, ++nw, n += tiles) {
    if (nw > 0) k = work_of(p, w_at);
    top = __int_as_float(0xff800000), sum = 0.0f;
    const float slope = a.slopes != nullptr && h < k.heads ? a.slopes[k.head0 + h] * kLog2e : 0.0f;
    for (int i = 0; i < tiles; ++i) {
      const int at = n + i, mask = at % kMasks;
      wait_or_stop_one(&sh.masks[mask], (at / kMasks) & 1, stop);  // giving up shows in `stop`
      if (!wait_or_stop(&sh.s_full[at & 7], (at >> 3) & 1, stop)) break;
      tc_fence_after();
      const uint32_t s_at = tmem + buf * kKeys + lanes;
      float z[kPart];
      float high = __int_as_float(0xff800000);
#pragma unroll
      for (int c = 0; c < kPart; c += kStep) {
        uint32_t v[kStep];
        tmem_ld(v, s_at + copy * kPart + c);
        const int e0 = copy * kPart + c;
        const uint32_t bits = (sh.seen[mask][e0 / 32] >> (e0 % 32)) & (kStep == 32 ? 0xffffffffu : 0xffffu);
        tmem_wait_ld(v);
        if (a.softcap > 0.0f) {
          // The second form only where a row of the warp needs it: logits are mostly
          // far below their cap (shared entries, 2048 rows x 512: 154 us, 178 with both).
          float most = 0.0f;
#pragma unroll
          for (int j = 0; j < kStep; ++j) most = fmaxf(most, fabsf(__uint_as_float(v[j])));
          const bool bent = __any_sync(0xffffffffu, most * fabsf(p.scale_over_cap) >= kBent);
          if (bent) {
#pragma unroll
            for (int j = 0; j < kStep; j += 2) {
              const uint64_t x = pair(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), u = mul2(x, twice(p.scale_over_cap));
              const float2 low = capped_low(x, u, scale);
              z[c + j] = low.x, z[c + j + 1] = low.y;
              const float2 high = capped_high(u, p.cap_log2e), at = both(u);
              if (!(fabsf(at.x) < kBent)) z[c + j] = high.x;
              if (!(fabsf(at.y) < kBent)) z[c + j + 1] = high.y;
            }
          } else {
#pragma unroll
            for (int j = 0; j < kStep; j += 2) {
              const uint64_t x = pair(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
              const float2 low = capped_low(x, mul2(x, twice(p.scale_over_cap)), scale);
              z[c + j] = low.x, z[c + j + 1] = low.y;
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < kStep; ++j) z[c + j] = __uint_as_float(v[j]) * scale;
        }
        if (a.slopes != nullptr) {
#pragma unroll
          for (int j = 0; j < kStep; ++j) z[c + j] += slope * sh.away[mask][e0 + j];
        }
        if (bits != (kStep == 32 ? 0xffffffffu : 0xffffu)) {
#pragma unroll
          for (int j = 0; j < kStep; ++j)
            if (((bits >> j) & 1) == 0) z[c + j] = __int_as_float(0xff800000);
        }
#pragma unroll
        for (int j = 0; j < kStep; ++j) high = fmaxf(high, z[c + j]);
      }
      // move the reference where the maximum has outgrown it
      if (__any_sync(0xffffffffu, high > top + kGrowth)) {
        const float moved = fmaxf(top, high);
        const float factor = is_low(moved) ? 1.0f : exp2_fast(top - moved);
        top = moved;
        sum *= factor;
        if (i > 0) {
          if (!wait_or_stop(&sh.pv_done[(at - 1) & 7], ((at - 1) >> 3) & 1, stop)) break;
          tc_fence_after();
          for (int c = 0; c < a.Dv; c += 16) {  // past Dv: columns that nothing reads, within the allocation
            uint32_t v[16];
            tmem_ld(v, tmem_o + lanes + c);
            tmem_wait_ld(v);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * factor);
            tmem_st(tmem_o + lanes + c, v);
          }
        }
      }
      const float ref = is_low(top) ? 0.0f : top;
      float part[4] = {};
#pragma unroll
      for (int j = 0; j < kPart; ++j) {
        z[j] = exp2_fast(z[j] - ref);
        part[j & 3] += z[j];
      }
      sum += (part[0] + part[1]) + (part[2] + part[3]);
      // the weights, over the scores: columns of the other copies' parts get zeros
#pragma unroll
      for (int c = 0; c < kKeys / 2; c += 16) {
        uint32_t v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int e = 2 * (c + j);  // first entry of column c + j
          if (COPIES == 1)
            v[j] = Pack<E>::two(z[e % kPart], z[e % kPart + 1]);
          else
            v[j] = e / kPart == copy ? Pack<E>::two(z[e % kPart], z[e % kPart + 1]) : 0u;
        }
        tmem_st(s_at + c, v);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sh.p_full[at & 7]);
      if (++buf == static_cast<uint32_t>(p.bufs)) buf = 0;
    }
    if (tiles > 0) wait_or_stop(&sh.pv_done[(n + tiles - 1) & 7], ((n + tiles - 1) >> 3) & 1, stop);
    tc_fence_after();
    const bool failed = *stop != 0;  // a wait ran out: the rows become NaN
    sh.top[threadIdx.x] = failed ? 0.0f : top;
    sh.sum[threadIdx.x] = failed ? __int_as_float(0x7fc00000) : sum;
    if (!kStay || cluster > 1) break;
    if constexpr (kStay) {
      // ---- end of a work: join the two copies, 32 columns at a time, and write ----
      softmax_sync();
      float all = sh.top[h], total = 0.0f;
      if (COPIES == 2) all = fmaxf(all, sh.top[kRows % 128 + h]);
#pragma unroll
      for (int c = 0; c < COPIES; ++c) {
        const float m = sh.top[c * kRows + h], l = sh.sum[c * kRows + h];
        total += l != l ? l : is_low(m) ? 0.0f : l * exp2_fast(m - all);
      }
      if (copy == 0 && a.lse != nullptr && h < k.heads) a.lse[k.row * a.Hq + k.head0 + h] = logsum(all, total);
      const float weight = total != total ? total : is_low(top) ? 0.0f : exp2_fast(top - all) * inverse(all, total);
      E* out = static_cast<E*>(a.out) + (k.row * a.Hq + k.head0 + h) * a.Dv;
      for (int c = 0; c < a.Dv; c += 32) {  // past Dv: columns that nothing reads, within the allocation
        uint32_t v[32] = {};
        if (tiles > 0) {
          tmem_ld(v, tmem_o + lanes + c);
          tmem_wait_ld(v);
          if (c + 32 >= a.Dv) {  // O is read: the next work may have it
            tc_fence_before();
            mbar_arrive(&sh.o_free);
          }
        }
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(v[j]) * weight;
        bool writes = true;
        if (COPIES == 2) {  // the copies write every other 32 columns, by way of two buffers
          float(&part)[36] = reinterpret_cast<AttParts*>(smem + p.parts_at)->part[(c >> 5) & 1][h & 63];
          writes = ((c >> 5) & 1) == copy;
          if (!writes) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<float4*>(&part[j]) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
          }
          softmax_sync();
          if (writes) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 y = *reinterpret_cast<const float4*>(&part[j]);
              x[j] += y.x, x[j + 1] += y.y, x[j + 2] += y.z, x[j + 3] += y.w;
            }
          }
        }
        if (writes && h < k.heads) {
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            if (c + j < a.Dv)
              *reinterpret_cast<uint4*>(out + c + j) =
                  make_uint4(Pack<E>::two(x[j], x[j + 1]), Pack<E>::two(x[j + 2], x[j + 3]),
                             Pack<E>::two(x[j + 4], x[j + 5]), Pack<E>::two(x[j + 6], x[j + 7]));
        }
      }
      softmax_sync();  // top and sum are read
    }
    }
  }

  // ---- join the copies ----
  // Every row of the buffer below is scaled to its head's maximum in this CTA.
  __syncthreads();
  if (*stop != 0) {  // a wait ran out: nobody may have waited for what is in flight
    if (one) mma_drain(&sh.drained[warp - kMmaWarp]);
    copy_commit();
    copy_wait<0>();
    __syncthreads();
  }
  if (!kStay || cluster > 1) {
  const int pad = p.v_blocks * 64 + 4;  // floats per row: rows 4 banks apart
  float* rows = reinterpret_cast<float*>(smem);
  if (warp < 4) {
    const int h = threadIdx.x % kRows;
    float all = sh.top[h], total = 0.0f;
#pragma unroll
    for (int c = 1; c < COPIES; ++c) all = fmaxf(all, sh.top[c * kRows + h]);
#pragma unroll
    for (int c = 0; c < COPIES; ++c) {
      const float m = sh.top[c * kRows + h], l = sh.sum[c * kRows + h];
      total += l != l ? l : is_low(m) ? 0.0f : l * exp2_fast(m - all);
    }
    if (threadIdx.x < kRows) {
      sh.head_top[h] = all;
      sh.head_sum[h] = cluster == 1 ? inverse(all, total) : total;
      if (cluster == 1 && a.lse != nullptr && h < k.heads) a.lse[k.row * a.Hq + k.head0 + h] = logsum(all, total);
    }
    const float weight = is_low(top) ? 0.0f : exp2_fast(top - all);
    const uint32_t lanes = static_cast<uint32_t>(warp) << 21;
    for (int c = 0; c < a.Dv; c += 32) {  // past Dv: columns that nothing reads, in the rows' padding
      uint32_t v[32] = {};
      if (tiles > 0) {
        tmem_ld(v, tmem_o + lanes + c);
        tmem_wait_ld(v);
      }
      float* dst = rows + threadIdx.x * pad + c;
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<float4*>(dst + j) =
            make_float4(__uint_as_float(v[j]) * weight, __uint_as_float(v[j + 1]) * weight,
                        __uint_as_float(v[j + 2]) * weight, __uint_as_float(v[j + 3]) * weight);
    }
  }
  tc_fence_before();
  __syncthreads();

  // ---- write, or join the CTAs first ----
  // Eight outputs per thread and step; a step of a warp takes as many whole
  // rows as fit its lanes (Dv <= 256: one at least).
  const int per_row = a.Dv / 8, at_once = 32 / per_row;
  const int sub_row = lane / per_row, c = (lane - sub_row * per_row) * 8;
  const int step = (kAttThreads / 32) * at_once;
  const int heads = k.heads;
  const int row0 = sub_row < at_once ? warp * at_once + sub_row : heads;
  E* out = static_cast<E*>(a.out) + (k.row * a.Hq + k.head0) * a.Dv;
  auto write = [&](int h, int c, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(out + static_cast<int64_t>(h) * a.Dv + c) =
        make_uint4(Pack<E>::two(x[0], x[1]), Pack<E>::two(x[2], x[3]), Pack<E>::two(x[4], x[5]), Pack<E>::two(x[6], x[7]));
  };
  auto add = [](float (&x)[8], float4 u, float4 v, float f) {
    x[0] += u.x * f, x[1] += u.y * f, x[2] += u.z * f, x[3] += u.w * f;
    x[4] += v.x * f, x[5] += v.y * f, x[6] += v.z * f, x[7] += v.w * f;
  };
  for (int h = row0; h < heads; h += step) {
    float x[8] = {};
#pragma unroll
    for (int q = 0; q < COPIES; ++q) {
      const float* from = rows + (q * kRows + h) * pad + c;
      add(x, *reinterpret_cast<const float4*>(from), *reinterpret_cast<const float4*>(from + 4), 1.0f);
    }
    if (cluster == 1) {
      const float f = sh.head_sum[h];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= f;
      write(h, c, x);
    } else {
      float* to = rows + h * pad + c;
      *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(to + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
  if (cluster > 1) {
    cluster_sync();
    const uint32_t top_addr = smem_addr(sh.head_top), sum_addr = smem_addr(sh.head_sum), rows_addr = smem_addr(rows);
    // four outputs per thread, all reads of all CTAs in flight together
    const int fours = a.Dv / 4, outputs = heads * fours;
    for (int i = static_cast<int>(rank) * kAttThreads + threadIdx.x; i < outputs; i += cluster * kAttThreads) {
      const int h = i / fours, c = (i - h * fours) * 4;
      float m[8], l[8], all = __int_as_float(0xff800000), total = 0.0f;
      float4 u[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const uint32_t from = r < cluster ? r : 0;
        m[r] = __uint_as_float(ld_dsmem_u32(map_rank(top_addr + 4 * h, from)));
        l[r] = __uint_as_float(ld_dsmem_u32(map_rank(sum_addr + 4 * h, from)));
        u[r] = ld_dsmem_f4(map_rank(rows_addr + 4 * (h * pad + c), from));
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) all = fmaxf(all, m[r]);
      float4 x = {};
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (r >= cluster) continue;
        const float f = is_low(m[r]) ? 0.0f : exp2_fast(m[r] - all);
        total += l[r] != l[r] ? l[r] : l[r] * f;
        x.x += u[r].x * f, x.y += u[r].y * f, x.z += u[r].z * f, x.w += u[r].w * f;
      }
      const float f = inverse(all, total);
      *reinterpret_cast<uint2*>(out + static_cast<int64_t>(h) * a.Dv + c) =
          make_uint2(Pack<E>::two(x.x * f, x.y * f), Pack<E>::two(x.z * f, x.w * f));
      if (c == 0 && a.lse != nullptr) a.lse[k.row * a.Hq + k.head0 + h] = logsum(all, total);
    }
    cluster_sync();  // the others may still read this CTA's rows
  }
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, p.tmem_cols);
  }
}

template <typename E, int COPIES>
topk_status launch_copies(const AttParams& p, int dev, int cluster, int64_t grid, size_t bytes, cudaStream_t stream) {
  constexpr auto kernel = attention_kernel<E, COPIES>;
  const topk_status st = allow_shared<kernel>(dev);
  if (st != TOPK_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kAttThreads);
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

template <typename E>
topk_status launch_typed(const sparse_attention_args& a, int dev, int sm_count, cudaStream_t stream) {
  AttParams p = {};
  p.a = a;
  p.heads = a.Hq / a.Hkv;
  p.m_tiles = p.heads / 128 + (p.heads % 128 != 0);
  p.scale_log2e = finite(static_cast<double>(a.scale) * kLog2e);
  if (a.softcap > 0.0f) {
    p.scale_over_cap = finite(static_cast<double>(a.scale) / a.softcap);
    p.cap_log2e = finite(static_cast<double>(a.softcap) * kLog2e);
  }
  p.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page_size == 1 << i) p.page_shift = i;
  p.pages = a.num_pages < INT32_MAX ? static_cast<uint32_t>(a.num_pages) : INT32_MAX;
  p.table_width = a.table_width < INT32_MAX ? static_cast<uint32_t>(a.table_width) : INT32_MAX;
  p.d_blocks = (a.D + 63) / 64;
  p.v_blocks = (a.Dv + 63) / 64;
  p.shared = a.k == a.v && a.Dv <= a.D && a.k_page_stride == a.v_page_stride && a.k_token_stride == a.v_token_stride &&
             a.k_head_stride == a.v_head_stride;
  p.q_vector = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && a.q_seq_stride % 8 == 0 && a.q_token_stride % 8 == 0 &&
               a.q_head_stride % 8 == 0;
  // As many copies as the heads leave room for: 64 rows x 2048 entries with 8
  // heads a key head take 92 us with 4 copies, 103 with 2, 142 with 1.
  const int copies = p.heads <= 32 ? 4 : p.heads <= 64 ? 2 : 1;
  // Shared memory: Q, then the ring; at the end the same bytes hold the rows
  // to be joined. Two CTAs share an SM where two stages each fit (and TMEM
  // holds both), else one CTA has as many stages as fit (64 rows x 2048 entries
  // x 8 key heads: 92 us with two, 109 with one).
  const int q_bytes = 128 * 128 * p.d_blocks;
  p.k_bytes = kKeys * 128 * p.d_blocks;
  p.v_bytes = p.shared ? 0 : kKeys * 128 * p.v_blocks;
  p.tmem_cols = copies == 4 && 2 * kKeys + p.v_blocks * 64 <= 256 ? 256 : 512;  // two CTAs or one on an SM
  p.bufs = (p.tmem_cols - p.v_blocks * 64) / kKeys < kMaxBufs ? (p.tmem_cols - p.v_blocks * 64) / kKeys : kMaxBufs;
  const int join = 128 * (p.v_blocks * 64 + 4) * 4;
  const int parts = copies == 2 ? static_cast<int>(sizeof(AttParts)) : 0;
  const int whole = kMaxShared - parts - static_cast<int>(sizeof(AttShared));
  const int half = kMaxShared / 2 - 1024 - static_cast<int>(sizeof(AttShared));
  const int least = p.shared ? 3 : 2;  // stages below which two CTAs gain nothing
  const bool two = copies == 4 && p.tmem_cols == 256 && q_bytes + least * (p.k_bytes + p.v_bytes) <= half && join <= half;
  int room = ((two ? half : whole) - q_bytes);
  int stages = room / (p.k_bytes + p.v_bytes);
  if (stages > kMaxStages) stages = kMaxStages;
  p.k_stages = stages;
  p.v_stages = p.shared ? 0 : stages;
  if (!p.shared && stages < kMaxStages && room - stages * (p.k_bytes + p.v_bytes) >= p.v_bytes) ++p.v_stages;
  p.k_at = q_bytes;
  p.v_at = q_bytes + p.k_stages * p.k_bytes;
  int operands = p.v_at + p.v_stages * p.v_bytes;
  if (operands < join) operands = (join + 15) / 16 * 16;
  p.parts_at = operands;
  p.shared_at = operands + parts;
  // CTAs of this kernel that share an SM must find their TMEM free: one that
  // waited for it could hold up its cluster, and that the CTA it waits for. So
  // those with all 512 columns take all of the shared memory, the others more
  // than a third.
  size_t bytes = static_cast<size_t>(operands) + parts + sizeof(AttShared);
  const size_t floor_bytes = p.tmem_cols == 512 ? kMaxShared : 77 * 1024;
  if (bytes < floor_bytes) bytes = floor_bytes;
  const int64_t work = static_cast<int64_t>(a.B) * a.T * a.Hkv * p.m_tiles;
  p.works = static_cast<uint32_t>(work);
  // Few rows: share each over the CTAs that would idle, down to two tiles each
  // (one row x 2048 entries, one key head: 25.5 us on one CTA, 16.9, 12.0 and
  // 9.8 on 2, 4 and 8; 16 key-head rows x 512: 8.4 us at two tiles a CTA, 9.4
  // at one and at four).
  const int64_t slots = static_cast<int64_t>(sm_count) * (two ? 2 : 1);
  const int tiles = tiles_of(a.K);
  int cluster = 1;
  while (cluster < 8 && work * cluster * 2 <= slots && cluster * 4 <= tiles) cluster *= 2;
  // One or two copies: CTAs stay, one on each place (2048 rows x 512 entries:
  // 131 us, 166 with a CTA a row, half of which begins and ends it).
  const int64_t grid = copies <= 2 && cluster == 1 && work > slots ? slots : work * cluster;
  if ((work / grid + 1) * tiles > INT32_MAX) return TOPK_EINVAL;  // a CTA counts its tiles
  if (copies == 4) return launch_copies<E, 4>(p, dev, cluster, grid, bytes, stream);
  if (copies == 2) return launch_copies<E, 2>(p, dev, cluster, grid, bytes, stream);
  return launch_copies<E, 1>(p, dev, cluster, grid, bytes, stream);
}

}  // namespace

topk_status launch_attention(const sparse_attention_args& a, int dev, int sm_count, cudaStream_t stream) {
  return a.type == SPARSE_BF16 ? launch_typed<__nv_bfloat16>(a, dev, sm_count, stream)
                               : launch_typed<__half>(a, dev, sm_count, stream);
}

}  // namespace tki
