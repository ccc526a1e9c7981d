// tc.cuh -- the sm_103a instructions the matrix products are built from:
// mbarriers with bounded waits, TMA tile loads, tcgen05 products and tensor
// memory.  Thin wrappers of the PTX instructions, one each.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace cr {
namespace tc {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// ---- mbarriers --------------------------------------------------------------------

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done;
}

// What a wait may last: kWaitTurns turns of kTurnCycles clock cycles, about half a
// second.  Time that the block is held off its SM ends one turn at most,
// however long it is, and so does going on on another SM, whose clock differs.
constexpr int kWaitTurns = 16;
constexpr unsigned long long kTurnCycles = 1ull << 26;

// Waits for the phase of `parity` to complete.  False if that took too long, or
// if another role of the block gave up (*gave_up set): the caller then leaves
// its loop.  A wait for many steps may take `more` turns.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* gave_up,
                                         int more = 0) {
  if (bar_try(bar, parity)) return true;
  long long start = clock64();
  int left = kWaitTurns + more;
  while (!bar_try(bar, parity)) {
    if (*gave_up) return false;
    if ((unsigned long long)(clock64() - start) > kTurnCycles) {
      if (--left < 0) {
        *gave_up = 1;
        return false;
      }
      start = clock64();
    }
  }
  return true;
}

// Polls for the phase, as long as a wait may last, whoever gave up.
__device__ __forceinline__ void bar_poll(uint32_t bar, uint32_t parity) {
  long long start = clock64();
  for (int left = kWaitTurns; !bar_try(bar, parity) && left >= 0;) {
    if ((unsigned long long)(clock64() - start) > kTurnCycles) --left, start = clock64();
  }
}

// Makes initialised barriers visible to the async proxy and to the cluster.
__device__ __forceinline__ void bar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- clusters -----------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Block `rank`'s shared memory at the place of this block's `addr`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// ---- TMA ----------------------------------------------------------------------------

// Loads the map's box at column x, row y to dst; bytes count on bar.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// ---- tensor memory and products -----------------------------------------------------

// Whole warp.  Writes the address of `cols` columns to shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t smem_out, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_out),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle, of a tile that TMA
// wrote with it: rows of 128 bytes, eight rows to a 1024-byte atom.
//   K-major  (a row holds 64 K values of one M or N index): stride = bytes
//            between groups of 8 rows; lead is not used.
//   MN-major (a row holds 64 M or N values of one K index): stride = bytes
//            between groups of 8 K indices, lead = bytes between blocks of 64
//            M or N indices.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(lead >> 4) << 16 |
         (uint64_t)(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// Instruction descriptor: bf16 operands, fp32 accumulator, M x N.
constexpr uint32_t product_desc(uint32_t m, uint32_t n, bool a_mn, bool b_mn) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (n >> 3) << 17 | (m >> 4) << 24;
}

// One thread: D (tensor memory) = A B + (accumulate ? D : 0), K = 16.
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t desc,
                                    bool accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(desc), "r"((uint32_t)accumulate)
      : "memory");
}

// Arrives on bar when this thread's products so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

// Whole warp: 32 columns of the warp's 32 lanes, one lane (row) a thread.  The
// wait is part of the instruction, so that no register is read too early.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32]; "
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
      "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
      "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
      "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
      "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// The same at two addresses, with one wait.
__device__ __forceinline__ void tmem_ld32x2(uint32_t addr, uint32_t addr2, float* v, float* v2) {
  uint32_t r[32], s[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64]; "
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, "
      "[%65]; "
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]),
      "=&r"(r[7]), "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]),
      "=&r"(r[14]), "=&r"(r[15]), "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]),
      "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23]), "=&r"(r[24]), "=&r"(r[25]), "=&r"(r[26]), "=&r"(r[27]),
      "=&r"(r[28]), "=&r"(r[29]), "=&r"(r[30]), "=&r"(r[31]), "=&r"(s[0]), "=&r"(s[1]), "=&r"(s[2]),
      "=&r"(s[3]), "=&r"(s[4]), "=&r"(s[5]), "=&r"(s[6]), "=&r"(s[7]), "=&r"(s[8]), "=&r"(s[9]),
      "=&r"(s[10]), "=&r"(s[11]), "=&r"(s[12]), "=&r"(s[13]), "=&r"(s[14]), "=&r"(s[15]), "=&r"(s[16]),
      "=&r"(s[17]), "=&r"(s[18]), "=&r"(s[19]), "=&r"(s[20]), "=&r"(s[21]), "=&r"(s[22]), "=&r"(s[23]),
      "=&r"(s[24]), "=&r"(s[25]), "=&r"(s[26]), "=&r"(s[27]), "=&r"(s[28]), "=&r"(s[29]), "=&r"(s[30]),
      "=&r"(s[31])
      : "r"(addr), "r"(addr2)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]), v2[i] = __uint_as_float(s[i]);
}

}  // namespace tc
}  // namespace cr
