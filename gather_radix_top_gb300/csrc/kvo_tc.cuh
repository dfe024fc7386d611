// Tensor-core building blocks (tcgen05, sm_103a): shared-memory matrix
// descriptors, the MMA and its completion, tensor memory, and waits that give
// up after a bounded time.
//
// Operand tiles in shared memory use the 128-byte swizzle: a tile is rows of
// 128 bytes, eight rows to a 1,024-byte group, and the 16-byte piece c of row
// r lies at piece c ^ (r % 8).
#pragma once

#include <cstdint>

#include "kvo.h"
#include "kvo_device.cuh"

namespace kvo {

// Byte offset of 16-byte piece c (0..7) of row r in a swizzled tile.
__host__ __device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t c) {
  return r * 128u + ((c ^ (r & 7u)) << 4);
}

// Descriptor of a swizzled tile at shared address `addr` (row 0 of the tile
// 1,024-byte aligned; `addr` may be advanced inside a row by multiples of 32
// bytes, or by whole 8-row groups).  `chunk` is the distance in bytes between
// 64-element pieces of the M or N dimension where that one is contiguous in
// memory; it is unused where K is.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t chunk) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(chunk >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor: fp32 accumulators, M = 128, N columns.
// operand: 1 = bf16 (kind::f16), 0 = e4m3 (kind::f8f6f4); the major flags say
// that the operand's M or N dimension, not K, is contiguous in memory.
__host__ __device__ constexpr uint32_t mma_desc(uint32_t operand, uint32_t n, bool a_mn_major, bool b_mn_major) {
  return 1u << 4 | operand << 7 | operand << 10 | (a_mn_major ? 1u << 15 : 0u) | (b_mn_major ? 1u << 16 : 0u) |
         (n >> 3) << 17 | (128u >> 4) << 24;
}

__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

// `bar` gets one arrival once every MMA this thread has issued is complete.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// One warp: `cols` (a power of two, 32..512) columns of tensor memory; the
// base address goes to *slot (shared memory).  No other CTA of the SM may
// hold columns that this one needs: the caller's shared memory sees to that.
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}

// 32 consecutive columns of the warp's 32 lanes (lane quadrant = warp % 4),
// one lane per thread.  tmem_ld_wait before the values are used.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_ld4(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_st4(uint32_t addr, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0, %1, %2, %3};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---- Two CTAs of a cluster (ranks 0 and 1) on one matrix product.  Rank 0
// issues the MMAs; operands and accumulators are at the same addresses in both.
// M is 256: a CTA holds 128 rows of A and of D (all N columns of them, in its
// tensor memory), and N / 2 rows of B.

__host__ __device__ constexpr uint32_t pair_desc(uint32_t operand, uint32_t n, bool a_mn_major, bool b_mn_major) {
  return (mma_desc(operand, n, a_mn_major, b_mn_major) & ~(31u << 24)) | (256u >> 4) << 24;
}

__device__ __forceinline__ void pair_mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// The barrier at this address in the CTAs of `mask` (bit r: rank r) gets one
// arrival once every pair MMA this thread has issued is complete.
__device__ __forceinline__ void pair_commit(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(mask)
      : "memory");
}

// One warp of each CTA, at the same time.
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void pair_tmem_free(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}

// An arrival at a barrier of another CTA of the cluster (or this one), given
// its cluster address, after this thread's accesses to its own CTA's memory: for
// operands there, which its own tensor core reads.  (An order over the whole
// cluster takes about 2,200 clocks.)
__device__ __forceinline__ void cluster_mbar_arrive_own(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// The same without an order: for accesses that are complete by themselves, as
// loads from tensor memory are once they have been waited for.
__device__ __forceinline__ void cluster_mbar_arrive_relaxed(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// `bytes` of this CTA's shared memory to another CTA's, given the cluster
// addresses of the destination and of a barrier there that it completes on.
__device__ __forceinline__ void bulk_copy_s2peer(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// A box of a three-dimensional tensor map to this CTA's shared memory at
// `dst`; completes on the barrier at cluster address `bar`, of either CTA.
__device__ __forceinline__ void pair_load_box(uint32_t dst, const void* map, int32_t x, int32_t y, int32_t z,
                                              uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// As if a copy of `bytes` that `bar` expects had come.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A CTA whose waits share `gave_up` (a shared-memory word).  Waits for phase
// `parity` of `bar`; after `clocks`, or as soon as another thread of the CTA
// has given up, it returns false.  What is in flight then is waited for once
// more before the CTA ends, with landed().
__device__ __forceinline__ bool wait_or_give_up(uint64_t* bar, uint32_t parity, volatile uint32_t* gave_up,
                                                long long clocks) {
  const uint32_t a = smem_u32(bar);
  uint32_t done;
  long long start = 0;
  for (uint32_t i = 0;; ++i) {
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(a), "r"(parity)
        : "memory");
    if (done) return true;
    if ((i & 15u) == 15u) {
      if (*gave_up) return false;
      const long long now = clock64();
      if (start == 0) start = now;
      if (now - start > clocks) {
        *gave_up = 1;
        return false;
      }
    }
  }
}

// Waits for a phase that work in flight completes, whether or not other
// waits have given up; false after about a second.
__device__ __forceinline__ bool landed(uint64_t* bar, uint32_t parity) {
  const long long start = clock64();
  while (!mbar_test(bar, parity))
    if (clock64() - start > KVO_WAIT_CLOCKS) return false;
  return true;
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts8(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}

// 16 bytes from global to shared memory without a register; zeros if !take.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, bool take) {
  const uint32_t bytes = take ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows r0..r3 of a two-dimensional tensor map whose box is one row of 128
// bytes, from element column `col`: 512 bytes of a swizzled tile at `dst`.
// Completes on `bar`.
__device__ __forceinline__ void gather_rows(uint32_t dst, const void* map, int32_t col, int32_t r0, int32_t r1,
                                            int32_t r2, int32_t r3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(col), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(smem_u32(bar))
      : "memory");
}

// The tensor map's box from element column `col` and row `row` on, as rows of
// 128 bytes of a swizzled tile at `dst`.  Completes on `bar`.
__device__ __forceinline__ void load_box(uint32_t dst, const void* map, int32_t col, int32_t row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(col), "r"(row), "r"(smem_u32(bar))
      : "memory");
}

// Barrier `id` (1..15) of `threads` threads of the CTA.
__device__ __forceinline__ void named_sync(uint32_t id, uint32_t threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace kvo
