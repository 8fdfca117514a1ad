// kvq_tc.cuh -- 5th-generation tensor core (tcgen05) helpers for sm_103a:
// TMEM allocation, shared-memory matrix descriptors, MMA issue/commit and
// TMEM <-> register moves, written as inline PTX.
#pragma once

#include <limits.h>
#include <stdint.h>

#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {

// Heaviest sequences first: CTA row z of the grid takes the sequence of
// rank z by 2 L - n (a proxy for its keys per query; for cross attention they
// are L), so the long prefixes
// start in the first wave and the short ones fill the tail.  Batches above
// 64 sequences keep their order.
__device__ __forceinline__ int heavy_first_sequence(const AttnParams& P, int z) {
  if (P.batch > 64) return z;
  const int lane = threadIdx.x & 31;
  int key[2], me = -1;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = lane + 32 * k;
    key[k] = INT_MIN;
    if (b < P.batch) key[k] = P.cross ? __ldg(P.seq_lens + b) : 2 * __ldg(P.seq_lens + b) - (__ldg(P.cu_q + b + 1) - __ldg(P.cu_q + b));
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = lane + 32 * k;
    int rank = 0;
    for (int j = 0; j < P.batch; ++j) {
      const int kj = __shfl_sync(0xffffffffu, key[j >> 5], j & 31);
      rank += (kj > key[k] || (kj == key[k] && j < b)) ? 1 : 0;
    }
    if (b < P.batch && rank == z) me = b;
  }
  const unsigned m = __ballot_sync(0xffffffffu, me >= 0);
  const int src = m ? __ffs(m) - 1 : 0;
  const int b = __shfl_sync(0xffffffffu, me, src);
  return m ? b : z;
}

namespace tc {

// 4-D tensor copy (TMA) of one box of `map` at coordinates (c0..c3) into
// shared memory, completion counted on `bar`.  `map` must live in the kernel
// parameter space (a __grid_constant__ parameter) or global memory; c0 times
// the element size must be a multiple of 16 bytes; rows outside the tensor
// arrive as zeros and still count as transaction bytes.
__device__ __forceinline__ void tma_load_4d(void* dst, const void* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "r"(smem_addr(bar))
      : "memory");
}

// Shared-memory matrix descriptor for a K-major operand stored in the
// canonical 128-byte-swizzle layout: rows of 128 bytes (64 fp16 along K),
// 8-row groups 1024 bytes apart, 16-byte chunk c of row r stored at chunk
// c ^ (r & 7).  The tile base must be 1024-byte aligned; a k-step of 16
// elements inside a 64-element atom advances the start address by 32 bytes.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFF) >> 4);  // start address >> 4
  d |= (uint64_t)1 << 16;                     // leading byte offset (unused for swizzled K-major)
  d |= (uint64_t)(1024 >> 4) << 32;           // stride byte offset: 8 rows x 128 B
  d |= (uint64_t)1 << 46;                     // descriptor version for tcgen05
  d |= (uint64_t)2 << 61;                     // 128-byte swizzle
  return d;
}

// Byte offset of (row, 16-byte chunk) inside one 64-element-wide atom.
__device__ __forceinline__ int sw128_off(int row, int chunk) { return row * 128 + 16 * (chunk ^ (row & 7)); }

// Instruction descriptor, kind::f16: fp16 A and B, fp32 accumulator, both K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void alloc(uint32_t* slot_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One lane of the warp, the same one each time; every lane calls these.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(is));
  return is;
}
// MMAs and commits issued by the lane whose `on` is set: the warp's control flow
// stays uniform, and descriptors in uniform registers.
// D[tmem] (+)= A[smem] . B[smem]^T.
__device__ __forceinline__ void mma_ss_if(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
// D[tmem] (+)= A[tmem] . B[smem]^T: A is M rows in TMEM lanes 0 .. M-1, each k-step
// of 16 elements in 8 consecutive 32-bit columns from `a` (element 2j in the low
// half of column j).
__device__ __forceinline__ void mma_ts_if(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
// Arrive on `bar` once all tcgen05 operations issued before by this lane complete.
__device__ __forceinline__ void commit_if(uint32_t on, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_addr(bar)),
      "r"(on)
      : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns (lane = TMEM row of this warp's quarter).
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// The registers a tcgen05.ld filled are final only after wait_ld: passing
// them through an empty volatile asm placed after the wait keeps the compiler
// from moving their uses above it.
template <int N>
__device__ __forceinline__ void regs_after_wait(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four 8x8 fp16 matrices from registers to shared memory, transposed: lane
// 8i + r gives the address of row r of matrix i as stored.
__device__ __forceinline__ void stsm_x4_t(uint32_t saddr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(saddr), "r"(r0), "r"(r1),
               "r"(r2), "r"(r3)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

}  // namespace tc
}  // namespace kvq
