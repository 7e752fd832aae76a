// Inline-PTX wrappers of the fifth-generation tensor cores (sm_103a): TMEM,
// tcgen05.mma with operands in shared memory or TMEM, its completion on
// mbarriers, and asynchronous 16-byte copies that feed it.
//
// Shared-memory operands use one layout throughout, the 128-byte swizzle:
// rows of 128 bytes (64 elements of 16 bits, 128 of 8), groups of 8 rows of
// 1024 bytes, the 16-byte unit j of row r stored at unit j ^ (r & 7).
#pragma once

#include <cuda.h>

#include <cstdint>

#include "ptx.cuh"

namespace tki {

// ---- TMEM -------------------------------------------------------------------

// One warp allocates `columns` (a power of two, 32 to 512) and writes the
// address to *dst; the same warp frees them.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Waits for this thread's TMEM loads: for uses of the values that are volatile
// assembly themselves, and so stay behind it.
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// The same for any use. `v` is an operand, so that nothing that
// uses the loaded values can move ahead of the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]),
                 "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]),
                 "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]),
                 "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]),
                 "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Columns [addr, addr + 16) or + 32 of this warp's 32 lanes, one lane per
// thread; the values are there after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld(uint32_t (&v)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld(uint32_t (&v)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// ---- matrix products --------------------------------------------------------

// Descriptor of a shared-memory operand in the layout above. `other` is the
// stride in bytes between 128-byte wide column blocks, which only an operand
// whose rows run along the product's inner dimension uses.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t other = 16) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (static_cast<uint64_t>(other >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: FP32 accumulators, M = 128 rows, N columns; `type`
// is 0 for fp16 (kind f16) and e4m3 (kind f8f6f4), 1 for bf16. With `b_rows`
// B's rows run along the inner dimension.
__device__ __forceinline__ constexpr uint32_t mma_desc(uint32_t type, uint32_t n, bool b_rows = false) {
  return (1u << 4) | (type << 7) | (type << 10) | (b_rows ? 1u << 16 : 0u) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// D[tmem] (+)= A[smem] B[smem], issued by one thread.
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(desc), "r"(add ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(desc), "r"(add ? 1u : 0u)
      : "memory");
}
// As mma_f16 with A in TMEM: row r in lane r, two elements per column.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(desc), "r"(add ? 1u : 0u)
      : "memory");
}

// Arrives on `bar` when every product this thread has issued is complete.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

// One thread of the (converged) warp: the one that issues products.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// ---- feeding ----------------------------------------------------------------

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// 16 bytes from global to shared memory, past L1: the first `bytes` (16 or 0)
// of them read, the rest zeros.
__device__ __forceinline__ void copy_bytes(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) { copy_bytes(dst, src, valid ? 16 : 0); }
// One arrival on `bar` when every copy16 of this thread so far is complete;
// it counts against the arrivals the barrier was initialised with.
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One box of a three-dimensional tensor map into shared memory; its bytes,
// also those outside the tensor, which arrive as zeros, count on `bar`.
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

// Byte offset of the 16-byte unit `unit` of row `row` within a 128-byte wide
// block in the layout above.
__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t unit) { return row * 128 + ((unit ^ (row & 7)) << 4); }

// As mbar_try_wait, without any sleep.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// How long a wait inside a kernel may take: a second, far beyond any real one,
// unless a test builds the kernels with less.
#ifndef SPARSE_WAIT_LIMIT_NS
#define SPARSE_WAIT_LIMIT_NS 1000000000
#endif
constexpr uint64_t kWaitLimit = SPARSE_WAIT_LIMIT_NS;
constexpr bool kNap = kWaitLimit >= 1000000;  // a look that sleeps may outlast a shorter limit

// Waits of the threads of one CTA on each other: false where it gave up. A
// wait that is not over in time raises `stop`, which ends every other wait of
// the CTA too; the caller then leaves its loop, but not the kernel before what
// it has in flight itself is complete.
__device__ __forceinline__ bool wait_or_stop_one(uint64_t* bar, uint32_t parity, volatile uint32_t* stop) {
  if (kNap ? mbar_try_wait(bar, parity) : mbar_test_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!(kNap ? mbar_try_wait_sleep(bar, parity, 20000u) : mbar_test_wait(bar, parity))) {
    if (*stop != 0) return false;
    if (global_timer_ns() - t0 > kWaitLimit) {
      *stop = 1;
      return false;
    }
  }
  return true;
}
// The same for a whole warp, with one answer for all of its lanes.
__device__ __forceinline__ bool wait_or_stop(uint64_t* bar, uint32_t parity, volatile uint32_t* stop) {
  return __all_sync(0xffffffffu, wait_or_stop_one(bar, parity, stop));
}

// Until every product that this thread has issued is complete, whatever was
// given up: their operands, sums and barriers may go away after it. `bar`
// is used for nothing else.
__device__ __forceinline__ void mma_drain(uint64_t* bar) {
  mma_commit(bar);
  mbar_wait_bounded(bar, 0, 1000000000ull);
}

}  // namespace tki
