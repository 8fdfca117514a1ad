// kvq_cross.cuh -- what the cross-attention kernels share: wide TMEM moves,
// MN-major operands, paired fp32 arithmetic, and rows added up in memory.
#pragma once

#include "kvq_common.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace tc {

// MN-major operand in 128-byte-swizzled lines of 64 elements along MN: groups of
// 8 lines along K 1024 bytes apart, the next 64 elements `lead` bytes further.
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr, int lead) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Four neighbouring fp32 values of global memory, each added to.
__device__ __forceinline__ void red_add4(float* p, float4 v) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// Two fp32 values at a time.
__device__ __forceinline__ uint64_t pair32(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair32(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 32 rows of D sums in TMEM (a lane each) go to `base`: the row at `to` (from
// base; none where negative) = (itself f + O) w.  Without `any` O is zeros,
// without `more` the row is; with `add` (f w = 1 in every lane) O w is added in
// memory, unread.  32 dims at a time through ADD_ROWS_BYTES of shared memory, so
// that a warp's stores and adds are whole 128-byte lines: four rows, eight lanes
// each.  Every lane calls it.
constexpr int ADD_ROWS_BYTES = 32 * 32 * 4;
template <int D>
__device__ __forceinline__ void add_rows(float* base, long long to, uint32_t o_tm, float f, float w, bool any, bool more,
                                         bool add, uint8_t* stage) {
  const int lane = threadIdx.x & 31;
  long long at[8];
  float rf[8], rw[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int row = 4 * k + (lane >> 3);
    at[k] = __shfl_sync(0xffffffffu, to, row);
    rf[k] = __shfl_sync(0xffffffffu, f, row);
    rw[k] = __shfl_sync(0xffffffffu, w, row);
  }
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    {
      uint32_t o[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = 0;
      if (any) {
        ld32(o_tm + c, o);
        wait_ld();
        regs_after_wait(o);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        sts128(stage + lane * 128 + 16 * ((j ^ lane) & 7), make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
    }
    __syncwarp();
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int row = 4 * k + (lane >> 3);
      x[k] = *reinterpret_cast<const float4*>(stage + row * 128 + 16 * ((lane ^ row) & 7));
    }
    __syncwarp();
    float* p = base + c + 4 * (lane & 7);
    if (add) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (at[k] >= 0) red_add4(p + at[k], make_float4(x[k].x * rw[k], x[k].y * rw[k], x[k].z * rw[k], x[k].w * rw[k]));
    } else {
      float4 e[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        e[k] = more && at[k] >= 0 ? __ldcg(reinterpret_cast<const float4*>(p + at[k])) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (at[k] >= 0)
          __stcg(reinterpret_cast<float4*>(p + at[k]),
                 make_float4(fmaf(e[k].x, rf[k], x[k].x) * rw[k], fmaf(e[k].y, rf[k], x[k].y) * rw[k],
                             fmaf(e[k].z, rf[k], x[k].z) * rw[k], fmaf(e[k].w, rf[k], x[k].w) * rw[k]));
    }
  }
}

}  // namespace tc
}  // namespace kvq
