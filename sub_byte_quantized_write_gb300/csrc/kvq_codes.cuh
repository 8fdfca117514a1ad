// kvq_codes.cuh -- rows of codes as fp16 operands of the tensor cores, shared by
// the kernels that expand them into shared memory.
#pragma once

#include "kvq_common.cuh"

namespace kvq {

// Two bf16 values (low half first) as an fp16 pair, rounded to nearest.  A
// bf16 value carries 8 significant bits, so the conversion is exact for 0 and
// for 2^-17 <= |x| <= 65504 (fp16 normals, and the subnormals that are
// multiples of 2^-24).  Smaller magnitudes round to a multiple of 2^-24
// (error at most 2^-25); magnitudes above 65504 become 65504 or infinity.
__device__ __forceinline__ uint32_t bf16x2_to_half2_bits(uint32_t w) {
  const __half2 hv = __floats2half2_rn(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return *reinterpret_cast<const uint32_t*>(&hv);
}

// Eight consecutive codes (head dims 8c .. 8c+7) of a raw row as four exact
// fp16 pairs of signed codes u - 2^(b-1) (INT8: as stored; FP8: the E4M3
// value; dense rows: the bf16 values), in dim order.  `one` 1: INT4 and INT2 codes
// one larger, u - 2^(b-1) + 1.
template <int MODE>
__device__ __forceinline__ uint4 codes8(const uint8_t* raw_row, int c, uint32_t one = 0) {
  uint32_t o[4];
  if constexpr (MODE == MODE_DBF16) {
    const uint4 w = *reinterpret_cast<const uint4*>(raw_row + 16 * c);
    o[0] = bf16x2_to_half2_bits(w.x);
    o[1] = bf16x2_to_half2_bits(w.y);
    o[2] = bf16x2_to_half2_bits(w.z);
    o[3] = bf16x2_to_half2_bits(w.w);
  } else if constexpr (MODE == MODE_INT4) {
    const uint32_t w = lds32(raw_row + 4 * c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = prmt(w, 0u, j | (4 << 4) | (j << 8) | (4 << 12));  // byte j in both halves
      o[j] = hsub2_bits(lop3_and_or(x, 0x00F0000Fu, 0x54006400u), 0x54806408u - one * 0x00100001u);
    }
  } else if constexpr (MODE == MODE_INT2) {
    const uint32_t w = *reinterpret_cast<const uint16_t*>(raw_row + 2 * c);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t x = prmt(w, 0u, j | (4 << 4) | (j << 8) | (4 << 12));
      o[2 * j] = hsub2_bits(lop3_and_or(x, 0x000C0003u, 0x5C006400u), 0x5C086402u - one * 0x00040001u);
      o[2 * j + 1] = hsub2_bits(lop3_and_or(x, 0x00C00030u, 0x4C005400u), 0x4C805420u - one * 0x00400010u);
    }
  } else if constexpr (MODE == MODE_F8T) {
    const uint2 w = make_uint2(lds32(raw_row + 8 * c), lds32(raw_row + 8 * c + 4));  // rows are D + 4 bytes
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = e4m3x2_to_half2_bits((j < 2 ? w.x : w.y) >> (16 * (j & 1)));
  } else {
    // INT8 channel rows (D bytes) are 8-byte aligned, token-head rows (D + 4) are not
    const uint2 w = MODE == MODE_INT8 ? lds64(raw_row + 8 * c)
                                      : make_uint2(lds32(raw_row + 8 * c), lds32(raw_row + 8 * c + 4));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t src = j < 2 ? w.x : w.y;
      const int bb = 2 * (j & 1);
      const uint32_t x = prmt(src, 0u, bb | (4 << 4) | ((bb + 1) << 8) | (4 << 12));
      o[j] = hsub2_bits(lop3_and_xor(x, 0x00FF00FFu, 0x64806480u), 0x64806480u);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace kvq
