// kvq_rope.cuh -- rotary positions: the angle of a (position, pair), its sine
// and cosine, and the turn of a row held by the lanes of a warp.
//
// Pair i of a row at position p turns by the angle p f_i: (a, b) becomes
// A (a c - b s, b c + a s) with c = cos(p f_i), s = sin(p f_i) and A a factor
// of its own (1, or what a scaled context asks for).
//
// Angles.  p f_i in fp32 is off by 2^-24 p f_i, 0.06 of a radian at a million
// positions, and fp64 runs at a small fraction of fp32's rate here.  So angles
// are counted in fixed point: u = f / (2 pi) turns as a 64-bit fraction, whole
// turns dropped; p u modulo 2^64 is the angle's fraction of a turn, exact but
// for p times u's own rounding (2^-64 for f below 2: below 2^-33 of a turn for
// any 32-bit p; 248 times that for the largest f, 2^16).  Its top 32 bits (cut at
// 2^-32 of a turn) give the quadrant and what is left of it, at most an
// eighth of a turn either way, where the Taylor series of sine (to y^9, the
// next term below 2e-9) and cosine (to y^10, below 2e-10) are as exact as
// fp32.
#pragma once

#include "kvq_common.cuh"

namespace kvq {

// inv_freq NULL: rows are not turned.
struct RopeArgs {
  const float* inv_freq;     // [rot / 2] radians per position
  const int32_t* positions;  // [num_tokens] or NULL: the positions of the write
  int rot, inter;            // dims that turn; 1: pairs (2i, 2i+1), 0: (i, i + rot / 2)
  float scale;
};

// f radians as a 64-bit fraction of a turn.  f = m 2^e with a 24-bit m, and
// 2^66 / (2 pi) as an integer (0.0151 above it): m times it is off by 2^24 *
// 0.0151 at most, which the shift by 2 - e (25 or more for f < 2) takes below one
// unit and that of the largest f, 2^16, to 247.
__device__ __forceinline__ uint64_t rope_turns(float f) {
  constexpr uint64_t C = 0xA2F9836E4E44152AULL;  // 2^66 / (2 pi) = 2^65 / pi
  const uint32_t bits = __float_as_uint(f);
  const int ex = (bits >> 23) & 255;
  const uint64_t m = (bits & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
  const int sh = 2 - ((ex ? ex : 1) - 150);  // right shift of m * C
  const uint64_t lo = m * C, hi = __umul64hi(m, C);
  uint64_t u;
  if (sh >= 64) u = sh >= 128 ? 0 : hi >> (sh - 64);
  else if (sh > 0) u = (hi << (64 - sh)) | (lo >> sh);
  else u = sh > -64 ? lo << -sh : 0;
  return (bits >> 31) ? 0 - u : u;
}

// (cos, sin) of position p, u turns per position.
__device__ __forceinline__ float2 rope_cos_sin(uint64_t u, int p) {
  const uint32_t ul = (uint32_t)u, uh = (uint32_t)(u >> 32);
  const uint32_t top = __umulhi(ul, (uint32_t)p) + uh * (uint32_t)p - (p < 0 ? ul : 0u);  // bits 32-63 of u * p
  const uint32_t quad = (top + 0x20000000u) >> 30;
  const float y = (float)(int32_t)(top - (quad << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float z = y * y;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);  // 1/9!, -1/7!
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -0.16666667f);
  s = fmaf(y * z, s, y);
  float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);  // -1/10!, 1/8!
  c = fmaf(z, c, -1.3888889e-3f);
  c = fmaf(z, c, 4.1666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.0f);
  const float a = (quad & 1) ? s : c, b = (quad & 1) ? c : s;
  return make_float2(__uint_as_float(__float_as_uint(a) ^ (((quad + 1) & 2) << 30)),
                     __uint_as_float(__float_as_uint(b) ^ ((quad & 2) << 30)));
}

// A row held by 32 lanes, lane l its elements l * EPL .. + EPL - 1 (EPL 2 or
// 4): the lane's factors, y = x c + partner s.  Pairs are whole multiples of 8
// elements apart, so a lane's partners are one lane's, or its own.
template <int EPL>
struct RopeLane {
  float c[EPL], s[EPL];
  int from;  // the lane that holds the partners
  bool on, inter;
};

template <int EPL, bool READ_ONLY>
__device__ __forceinline__ RopeLane<EPL> rope_lane(const RopeArgs& R, int pos, int lane) {
  RopeLane<EPL> r;
  const int d0 = lane * EPL, half = R.rot / 2;
  r.from = lane;
  r.inter = R.inter != 0;
  r.on = d0 < R.rot;
  if (r.on) {
    if (r.inter) {
#pragma unroll
      for (int e = 0; e < EPL; e += 2) {
        const float2 w = rope_cos_sin(rope_turns(load_input<READ_ONLY>(R.inv_freq + (d0 + e) / 2)), pos);
        r.c[e] = r.c[e + 1] = w.x * R.scale;
        r.s[e + 1] = w.y * R.scale;
        r.s[e] = -r.s[e + 1];
      }
    } else {
      const bool first = d0 < half;
      r.from = first ? lane + half / EPL : lane - half / EPL;
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        const float2 w = rope_cos_sin(rope_turns(load_input<READ_ONLY>(R.inv_freq + (first ? d0 : d0 - half) + e)), pos);
        r.c[e] = w.x * R.scale;
        r.s[e] = first ? -w.y * R.scale : w.y * R.scale;
      }
    }
  }
  return r;
}

// Turns a row; every lane of the warp calls this.  Dims past R.rot stay as they are.
template <int EPL>
__device__ __forceinline__ void rope_row(const RopeLane<EPL>& r, float (&x)[EPL]) {
  float o[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) {
    const float far = __shfl_sync(0xffffffffu, x[e], r.from);
    o[e] = r.inter ? x[e ^ 1] : far;
  }
  if (!r.on) return;
#pragma unroll
  for (int e = 0; e < EPL; ++e) x[e] = fmaf(x[e], r.c[e], o[e] * r.s[e]);
}

}  // namespace kvq
