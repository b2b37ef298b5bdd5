// Device-side building blocks of the tensor-core kernels: clusters of two
// CTAs, tensor copies that signal the leader's barrier, tcgen05 products with
// accumulators in tensor memory, and the shared-memory descriptors.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "rn_device.cuh"

namespace rn {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The cluster's barrier, and its two halves: what a thread does between them is
// ordered neither way.  Another CTA's shared memory may be touched only after
// a barrier of the whole cluster: until then that CTA need not have started.
// The instructions are the warp's (.aligned), so its lanes come together first:
// the code in front often ends with a branch of one lane.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

// the same shared-memory address in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// An arrival without release: what it hands on is tensor memory, whose reads
// have completed (tcgen05.wait::ld).  A release would first wait for the global
// stores of the same thread.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// brings a tensor map (a kernel argument) in before its first copy
__device__ __forceinline__ void prefetch_map(const CUtensorMap* tm) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(tm) : "memory");
}

// mbar_wait of a converged warp: every lane gets the same answer
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, unsigned* err, unsigned code) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, err, code));
}

// The instructions below that one thread has to issue are called by a whole
// converged warp, one elected lane of which issues them: their operands then
// stay in uniform registers (from inside a branch on the lane they had to be
// moved there one by one, which cost a quarter of the products' rate).

// 2-D tensor copy into this CTA's shared memory; `bar` may be the barrier of
// the cluster's other CTA.  x * element size must be a multiple of 16.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* tm, int x, int y,
                                            uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
      "l"(tm), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mbar_expect_elected(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}

// tensor memory: 512 columns (all of it) for the CTA pair; executed by one
// whole warp of each CTA
__device__ __forceinline__ void tmem_alloc_all(uint32_t smem_dst) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_dst)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}

__device__ __forceinline__ void tmem_free_all(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr));
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D (tensor memory) = A B (+ D): bf16 operands in shared memory of both CTAs
__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                              bool add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

// one arrival on the barrier at `bar` in each CTA of `mask` once every product
// the elected thread issued so far has completed
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t mask) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n\t}" ::"r"(bar),
      "h"((uint16_t)mask)
      : "memory");
}

// 32 lanes x 32 columns of fp32 from tensor memory: thread = lane
__device__ __forceinline__ void tmem_load32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_load_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Shared-memory matrix descriptors, 128-byte swizzle (atoms of 8 x 128 bytes,
// 1024-byte aligned).  K-major: the 128 bytes run along the reduction, the
// 8-row groups stand 1024 bytes apart, 16 reduction elements are 32 bytes.
// MN-major: the 128 bytes (64 elements) run along the rows of the result, the
// groups of 8 reduction elements stand 1024 bytes apart, the blocks of 64
// result rows 8192 bytes (64 reduction elements a stage), and 16 reduction
// elements are 2048 bytes.
constexpr uint64_t kDescBase = (1ull << 46) | (2ull << 61) | (64ull << 32);
constexpr uint64_t kDescK = kDescBase | (1ull << 16);
constexpr uint64_t kDescMN = kDescBase | (512ull << 16);

__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool mn) {
  return (mn ? kDescMN : kDescK) | (uint64_t)((addr & 0x3FFFFu) >> 4);
}
// descriptor step of 16 reduction elements
__device__ __forceinline__ uint64_t smem_desc_step(bool mn) { return mn ? 128 : 2; }

// Instruction descriptor: bf16 x bf16 -> fp32, M = 256 (the pair), N = 256
constexpr uint32_t kIdesc256 = (1u << 4) | (1u << 7) | (1u << 10) | ((256u >> 3) << 17) | ((256u >> 4) << 24);
constexpr uint32_t kIdescAMN = 1u << 15, kIdescBMN = 1u << 16;

}  // namespace rn
