// rr_tcgen05.cuh -- PTX wrappers of the fifth-generation tensor cores
// (tcgen05: tensor memory, block-scaled products, scale copies) and of tiled
// tensor copies, for the microscaled 4-bit product.
#pragma once

#include <cuda.h>

#include "rr_device.cuh"

namespace rr {

// One lane of a converged warp, the same one every time.  Tensor instructions
// take their operands from uniform registers: a loop that the whole warp runs,
// with only the instructions themselves under this predicate, keeps them there
// (in a loop that one lane runs alone every instruction took about 75 cycles to
// issue, and a product of 8192^3 1.5 times as long).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
// A value that is the same in all lanes, as one the compiler knows to be.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// --------------------------------------------------------------------------
// tensor memory
// --------------------------------------------------------------------------

// G: CTAs that work on one tile (cta_group), 1 or 2; the same for every call of
// a kernel.  With 2, both CTAs allocate and free, one of them issues the rest.

// Whole warp.  Writes the address of `columns` (a power of two, 32 .. 512)
// fresh columns to *slot.
template <int G>
__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t columns) {
  if constexpr (G == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
}
template <int G>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  if constexpr (G == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}

__device__ __forceinline__ void tcgen05_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tcgen05_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrives on `bar` (with G = 2, on that barrier of both CTAs) when every tensor
// operation this thread issued has completed.
template <int G>
__device__ __forceinline__ void tcgen05_commit(uint64_t *bar) {
  if constexpr (G == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// 32 lanes (this warp's quarter) by 32 columns of accumulators.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t r[32]) {
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
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t r[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// --------------------------------------------------------------------------
// shared-memory matrix descriptors: bits 0-13 start / 16, 16-29 leading-dimension
// byte offset / 16, 32-45 stride byte offset / 16, 46-47 version (1), 61-63 swizzle
// --------------------------------------------------------------------------

// A K-major operand tile of 128-byte rows with the 128-byte swizzle: groups of
// eight rows are 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t smem) {
  return (uint64_t)((smem >> 4) & 0x3fff) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// An unswizzled column of 16-byte rows (one scale atom: 32 rows): groups of
// eight rows are 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t smem) {
  return (uint64_t)((smem >> 4) & 0x3fff) | (1ull << 16) | (8ull << 32) | (1ull << 46);
}

// One scale atom (128 rows by 4 blocks, 512 bytes) to four columns of tensor
// memory, the same in the lanes of all four warps.
// With G = 2 in both CTAs, each from its own shared memory.
template <int G>
__device__ __forceinline__ void scale_copy(uint32_t tmem, uint64_t desc) {
  if constexpr (G == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// Instruction descriptor of a block-scaled 4-bit product (E2M1 by E2M1 with
// E8M0 scales, both operands K-major): bits 4-5 / 29-30 the first scale byte
// of B / A in each 32-bit column (0 or 2), 7-9 and 10-11 the element formats
// (1: E2M1), 17-22 N / 8, 23 the scale format (1: E8M0), 27-28 M / 128.
__device__ __forceinline__ constexpr uint32_t mx4_scale_at(int byte) {
  return ((uint32_t)byte << 4) | ((uint32_t)byte << 29);
}
__device__ __forceinline__ constexpr uint32_t mx4_instr_desc(int M, int N, int scale_at) {
  return mx4_scale_at(scale_at) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 7) << 27);
}

// D += A B^T over 64 elements of K (two scale blocks); accumulate false: D = A B^T.
// With G = 2 each CTA holds its half of the rows of D and A and of the columns
// of B, and the scales of its rows of A and of all columns of B.
template <int G>
__device__ __forceinline__ void mx4_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t scale_a,
                                        uint32_t scale_b, bool accumulate) {
  if constexpr (G == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(scale_a), "r"(scale_b), "r"((uint32_t)accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(scale_a), "r"(scale_b), "r"((uint32_t)accumulate)
        : "memory");
}

// --------------------------------------------------------------------------
// tiled tensor copies
// --------------------------------------------------------------------------

// Box of the two-dimensional map at (x bytes, row y); x is a multiple of 16.
__device__ __forceinline__ void tensor_load(void *smem_dst, const CUtensorMap *map, int x, int y, uint64_t *bar,
                                            uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_addr(smem_dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar)), "l"(pol)
      : "memory");
}
// The same where the bytes count on a barrier of either CTA of a pair (a
// cluster address).
__device__ __forceinline__ void tensor_load_pair(void *smem_dst, const CUtensorMap *map, int x, int y,
                                                 uint32_t cluster_bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_addr(smem_dst)),
      "l"(map), "r"(x), "r"(y), "r"(cluster_bar), "l"(pol)
      : "memory");
}
// Box of a three-dimensional map.
__device__ __forceinline__ void tensor_load_pair(void *smem_dst, const CUtensorMap *map, int x, int y, int z,
                                                 uint32_t cluster_bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint "
      "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_addr(smem_dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(cluster_bar), "l"(pol)
      : "memory");
}
__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// --------------------------------------------------------------------------
// clusters
// --------------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The cluster address of this CTA's shared-memory object in CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// 16 bytes to another CTA's shared memory.
__device__ __forceinline__ void cluster_store4(uint32_t cluster_addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

}  // namespace rr
