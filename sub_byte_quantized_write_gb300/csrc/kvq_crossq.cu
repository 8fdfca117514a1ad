// kvq_crossq.cu -- cross attention over quantised pages on the 5th-generation
// tensor cores (tcgen05, TMEM).
//
// The same sums as kvq_cross16.cu, with rows k_j = s_j c_j + z_j (inverse RHT
// after that) held as codes c_j: for a query rotated like the rows, q' = H (d q),
//   logit = scale (s_j (q' . c_j) + z_j sum(q')) / D
//   out   = d H ( sum_j (p_j s_j) c_j + sum_j p_j z_j ) / (D sum_j p_j)
// so that the tensor cores see the codes alone, exact small numbers in fp16.
// q' and p s are two fp16 terms each (22 bits).  8 D multiplies per (query, q
// head, key) for the 4 D of the exact products.
//
// Design: one CTA of 20 warps per (128 rows, kv head, sequence, part of the
// keys); a row is a (query, q head of the GQA group) pair; key tiles of 128, in
// two halves for the softmax.
//   warp 0      TMEM, and every tcgen05.mma: S = Q_hi C^T + Q_lo C^T (queries in
//               TMEM) and, half by half, O += P_hi V + P_lo V.  S(v + 1) is under
//               way while tile v is in its softmax.
//   warp 1      bulk copies of the raw page chunks, and the tiles' scales and zero
//               points in fp32.  K and V have places of their own, so that K runs
//               a tile ahead (together: 812 us for 726, see below).
//   warps 2, 3  codes to fp16 in the 128-byte swizzle.  V stays as it lies (an
//               MN-major operand): K and V are expanded alike and nothing is
//               transposed.
//   warps 4-19  softmax, a thread per row and half a tile: four groups of four
//               warps take the halves in turn.  They agree on the running maximum,
//               each publishing it for the next as soon as its half's is known,
//               and keep sums of their own, joined at the end.  (Two groups with
//               whole tiles, 128 logits to a thread: as fast, and more spills.)
// The queries' transform and the outputs' are made by the softmax threads, 32
// dims of a row each, in registers: by a warp to a row a CTA's start and end took
// 26 us of it.  The start and the end are fetched from L2 as instructions, some 5
// us each: they are written for few instructions.
// The reference that p is counted from follows the largest p s of the row so far
// (the running maximum of the logit plus the scale's exponent) and keeps it at
// 2^CQ_BASE .. 2^(CQ_BASE + CQ_SLACK), within fp16's range: a row of large values
// does not push the weights of others that the query looks at among the
// subnormals.  O is rescaled when the reference moves, which with a slack of 2^4
// was 8% of the call.  Every CQ_FLUSH tiles O is added in fp32 to the row where
// it will end up, since the accumulators truncate (kvq_cross16.cu): an error of
// 3e-6 to 8e-6 of an output over 8192 keys at 16 tiles; 8 would halve it for 7% of
// the time.  (Added by the last group, beside the next tile's softmax: 746 us for
// 713, measured before the reference went by p s.)  For the same
// reason value codes of odd keys are counted from 2^(b-1) - 1 and of even ones from
// 2^(b-1): from 2^(b-1) alone their mean is half a code, whose sum, which the zero
// points' then cancels, was many times the output's own and what it lost 1.2e-4
// (2-bit) and 1.6e-5 (4-bit) of an output over 8192 keys.
// Measured: 16 prompts of 101 .. 700 queries over 500 .. 4000 keys (4-bit, 32 q
// and 8 kv heads of 128): 737 us (the prefill kernel's form of it: 1024; with a
// factor by the largest scale so far: 713), 36% of the tensor cores' rate counting
// the doubled products.  What bounds it is the
// chain of a tile: logits from TMEM, maximum, weights, back, P.V, next S, some
// 8500 cycles with two tiles in flight (TMEM is full: S twice, O and Q; Q's terms
// in shared memory would make room for a third, which was not tried).
// (S half by half, each right after the P.V that frees its place: 721 us for 713.)
// Every wait is bounded; on a timeout the CTA reports KVQ_DEVERR_TIMEOUT, drains,
// frees its TMEM and returns.
//
// Sources: FastDeploy PR #7718 "Optimize AppendAttention for discrete head-wise
// block_idx" (head-wise tables, -1 sentinel); vllm-ascend-quantized-kv-cache
// METADATA, 运行机制 (paged cache read and dequantised).

#include <math_constants.h>

#include "kvq_codes.cuh"
#include "kvq_cross.cuh"
#include "kvq_decode.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int CQ_ROWS = PREFILL_ROWS;
constexpr int CQ_KT = 128, CQ_HALF = CQ_KT / 2;  // keys of a tile, and of a softmax step
constexpr int CQ_THREADS = 640;
constexpr int CQ_GROUPS = 4;  // of four softmax warps
constexpr int CQ_MMA_WARP = 0, CQ_COPY_WARP = 1, CQ_PROD_WARP = 2, CQ_PRODUCERS = 2, CQ_SOFTMAX_WARP = 4;
constexpr float CQ_BASE = 6.0f, CQ_SLACK = 8.0f;
constexpr int CQ_FLUSH = 16;  // (even: the same softmax group does it each time)
constexpr uint32_t CQ_NAP = 20;

template <int MODE, int D>
struct CqCfg {
  static constexpr int DATA = data_bytes(MODE, D);  // (scale and zero point follow)
  static_assert(DATA <= row_bytes_of(MODE, D), "the pad follows the codes");
  static constexpr int R = row_bytes_of(MODE, D);
  static constexpr int CHUNK = 16 * R;
  static constexpr int RAW = CQ_KT * R;           // raw rows of K (or V) of a tile
  static constexpr int HALF = CQ_KT * 128;        // 64 dims of 128 rows
  static constexpr int TILE = (D / 64) * HALF;    // fp16 K (or V) tile
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + 2 * TILE;
  static constexpr int OFF_RAW = OFF_V + 2 * TILE;           // [2][K, V][RAW]
  static constexpr int OFF_SC = OFF_RAW + 4 * RAW;           // [4, of tile v & 3][ks, kz, vs, vz, exponent of vs][128] f32
  // at the start [4 groups][128] sum, largest; at the end [4 groups][reference, l, pz][128] and what the rows hold
  static constexpr int OFF_SUM = OFF_SC + 4 * 5 * CQ_KT * 4;
  static constexpr int OFF_FAC = OFF_SUM + (3 * CQ_GROUPS + 1) * CQ_ROWS * 4;  // factors of a query's and of an output's dims [D] f32
  static constexpr int OFF_M = OFF_FAC + 2 * D * 4;          // [4 groups][128] published references
  static constexpr int OFF_BAR = OFF_M + CQ_GROUPS * CQ_ROWS * 4;
  static constexpr int NBAR = 48;
  static constexpr int PIECES = D / 32;  // of a row at the start and at the end: 32 dims, one thread
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;        // TMEM address, abort, sequence, [8] masks
  static constexpr int SMEM = OFF_MISC + 48 + 1024;
  // TMEM columns: S of tiles v & 1 (P over it: high terms, then low terms), O, Q high, Q low
  static constexpr int TM_O = 2 * CQ_KT, TM_QHI = TM_O + D, TM_QLO = TM_QHI + D / 2;
  static_assert(CQ_ROWS * D * 4 <= 4 * TILE, "the rows fit the K / V stages");
  static_assert(SMEM <= 232448, "shared memory");
};

// PFULL and PVDONE: weights, and their P.V, of half i of tile v, at 2 (v & 1) + i;
// PUB: group g, rows 32 q .. + 31, at 4 g + q; MEET: the groups' warps of rows 32 q
enum { QB_RAWKFULL = 0, QB_RAWKEMPTY = 2, QB_KFULL = 4, QB_KEMPTY = 6, QB_VFULL = 8, QB_VEMPTY = 10, QB_SFULL = 12,
       QB_PFULL = 14, QB_PVDONE = 18, QB_ODONE = 22, QB_DRAIN = 23, QB_PUB = 24, QB_MEET = 40,
       QB_RAWVFULL = 44, QB_RAWVEMPTY = 46 };

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }  // -126 <= e <= 127
// Hadamard transform of a thread's values.
template <int N>
__device__ __forceinline__ void wht_regs(float (&x)[N]) {
#pragma unroll
  for (int s = 1; s < N; s <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(i & s)) {
        const float a = x[i], b = x[i + s];
        x[i] = a + b;
        x[i + s] = a - b;
      }
}

__host__ __device__ constexpr uint32_t idesc_f16_mn(int M, int N, bool b_mn) {
  return tc::idesc_f16(M, N) | ((b_mn ? 1u : 0u) << 16);
}

}  // namespace

template <int MODE, int D>
__global__ void __launch_bounds__(CQ_THREADS, 1) crossq_kernel(const __grid_constant__ AttnParams P) {
  using C = CqCfg<MODE, D>;
  constexpr bool SCALES = MODE != MODE_INT8, ZEROS = SCALES && !byte_token_head(MODE);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (P.splits > 1) allow_dependent_launch();  // the join of the parts may launch; it waits for this grid
  const int h = blockIdx.y;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 4);
  int* seq_slot = reinterpret_cast<int*>(sm + C::OFF_MISC + 8);
  volatile int* mask = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 16);  // [8], of tile v & 7
  if (warp == CQ_COPY_WARP) {
    const int b0 = heavy_first_sequence(P, blockIdx.z);
    if (lane == 0) *seq_slot = b0;
  } else if (tid == 0) {
    for (int i = 0; i < C::NBAR; ++i) {
      const bool weights = (i >= QB_PFULL && i < QB_PFULL + 4) || (i >= QB_MEET && i < QB_MEET + 4);
      const bool producers = i == QB_RAWKEMPTY || i == QB_RAWKEMPTY + 1 || i == QB_VFULL || i == QB_VFULL + 1 || i >= QB_RAWVEMPTY;
      const bool k = i == QB_KFULL || i == QB_KFULL + 1;  // (and the scales)
      mbar_init(bar + i, k ? CQ_PRODUCERS + (SCALES ? 1 : 0) : producers ? CQ_PRODUCERS : weights ? 4 : 1);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  __syncthreads();
  const int b = *seq_slot;
  const int sp = blockIdx.x % P.splits, qtile = blockIdx.x / P.splits;
  const int G = P.group, Hq = P.num_q_heads, Hkv = P.num_kv_heads, bs = P.block_size, QB = CQ_ROWS / G;
  const int cq0 = __ldg(P.cu_q + b);
  int n = __ldg(P.cu_q + b + 1) - cq0;
  const bool first = tid == 0 && qtile == 0 && h == 0 && sp == 0;
  if (first && (n > P.max_q_per_seq || (n > 0 && (cq0 < 0 || cq0 > P.total_q - n)))) flag_error(P.dev_error, DEVERR_SEQ_LEN);
  n = min(n, P.max_q_per_seq);
  const int q0 = qtile * QB;
  if (q0 >= n || cq0 < 0) return;
  n = min(n, P.total_q - cq0);  // rows past the q that was given are neither read nor written
  if (q0 >= n) return;
  const int nq = min(QB, n - q0);
  int L = __ldg(P.seq_lens + b);
  if (L < 0 || L > P.max_blocks * bs) {
    if (first) flag_error(P.dev_error, L < 0 ? DEVERR_SEQ_LEN : DEVERR_TABLE_RANGE);
    L = L < 0 ? 0 : P.max_blocks * bs;
  }
  const int n_total = L / CQ_KT + (L % CQ_KT ? 1 : 0);  // (L may be next to 2^31)
  const int v0 = (int)((long long)sp * n_total / P.splits);
  const int nv = (int)((long long)(sp + 1) * n_total / P.splits) - v0;

  if (warp == CQ_MMA_WARP) {
    tc::alloc(tmem_slot, 512);
    tc::fence_before();
  }
  // the rows' queries into the K and V stages, 16-byte pieces XOR-swizzled by row (rows without one: zeros)
  const int piece_log2 = (D == 128 ? 4 : 3) + (P.dtype == DT_F32 ? 1 : 0);  // of a row
  for (int i = tid; i < CQ_ROWS << piece_log2; i += CQ_THREADS) {
    const int row = i >> piece_log2, at = i & ((1 << piece_log2) - 1), qi = cq0 + q0 + row / G;
    const bool is = row / G < nq && KVQ_IN_BOUNDS(qi < P.total_q, P.dev_error);
    const char* from = static_cast<const char*>(P.q) + (is ? ((((size_t)qi * Hq + h * G + row % G) << piece_log2) + at) * 16 : 0);
    cp_async16(sm + C::OFF_K + (((row << piece_log2) + (at ^ (row & 7))) << 4), from, is ? 16 : 0);
  }
  cp_async_commit();
  // factors: of a query's dims before the transform, of an output's after it
  const bool rht = MODE != MODE_INT8 && P.signs;
  float* qfac = reinterpret_cast<float*>(sm + C::OFF_FAC);
  float* ofac = qfac + D;
  if (tid < D) {
    float f = 1.0f, g = 1.0f;
    if constexpr (MODE == MODE_INT8) {
      f = __fdiv_rn(P.ch_amax[(size_t)h * D + tid], 127.0f);
      g = __fdiv_rn(P.ch_amax[((size_t)Hkv + h) * D + tid], 127.0f);
    } else if (rht) {
      f = __ldg(P.signs + tid) < 0 ? -1.0f : 1.0f;
      g = f / (float)D;
    }
    qfac[tid] = P.softmax_scale < 0.0f ? -f : f;  // (a negative scale is carried by the query)
    ofac[tid] = g;
  }
  cp_async_wait<0>();
  __syncthreads();
  // The rows' queries, rotated, scaled so that the largest element is 2^10 ..
  // 2^11, as two fp16 terms in TMEM.  A thread makes 32 dims of a row: piece g of
  // the transform is that of the pieces' sum with the signs of row g of the small
  // Hadamard matrix, so no thread needs another's.  (A
  // warp to a row, with shuffles: 12 us of a CTA's start.)
  const int g = (warp - CQ_SOFTMAX_WARP) >> 2, quad = warp & 3, r = 32 * quad + lane;  // (of the softmax warps)
  const uint32_t lanes = (uint32_t)(quad * 32) << 16;
  const bool real = r / G < nq;
  const bool softmax = warp >= CQ_SOFTMAX_WARP, has_piece = softmax && g < C::PIECES;
  float rb = 0.0f, rho = 0.0f;
  {
    float x[32];
    float2* meet = reinterpret_cast<float2*>(sm + C::OFF_SUM);
    if (has_piece) {
      float sum = 0.0f, amx = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = 0.0f;
      const uint8_t* row = sm + C::OFF_K + ((r << piece_log2) << 4);
#pragma unroll 1
      for (int k = rht ? 0 : g; k < (rht ? C::PIECES : g + 1); ++k) {
        const float sg = rht && (__popc(g & k) & 1) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float4 a;
          if (P.dtype == DT_F32) {
            a = *reinterpret_cast<const float4*>(row + (((8 * k + i / 4) ^ (r & 7)) << 4));
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(row + (((4 * k + i / 8) ^ (r & 7)) << 4) + 2 * (i & 4));
            a = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
          }
          const float4 f = *reinterpret_cast<const float4*>(qfac + 32 * k + i);
          x[i] = fmaf(sg * f.x, a.x, x[i]);
          x[i + 1] = fmaf(sg * f.y, a.y, x[i + 1]);
          x[i + 2] = fmaf(sg * f.z, a.z, x[i + 2]);
          x[i + 3] = fmaf(sg * f.w, a.w, x[i + 3]);
        }
      }
      if (rht) wht_regs<32>(x);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        sum += x[i];
        amx = fmaxf(amx, fabsf(x[i]));
      }
      meet[g * CQ_ROWS + r] = make_float2(sum, amx);
    }
    __syncthreads();
    tc::fence_after();
    if (softmax) {
      float sum = 0.0f, amx = 0.0f;
#pragma unroll
      for (int k = 0; k < C::PIECES; ++k) {
        const float2 o = meet[k * CQ_ROWS + r];
        sum += o.x;
        amx = fmaxf(amx, o.y);
      }
      const float scl = pow2(min(10 - (amx > 0.0f ? (int)(__float_as_uint(amx) >> 23) - 127 : 0), 100));
      const float sabs = fabsf(P.softmax_scale) * 1.4426950408889634f / (rht ? (float)D : 1.0f);
      rb = fmaxf(sabs / scl, 1e-30f);  // logit in log2 units: rb (s c.q'' + rho z)
      rho = sabs * sum / rb;
      if (has_piece) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float a = x[2 * j] * scl, e = x[2 * j + 1] * scl;
          hi[j] = pack_half2(a, e);
          const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&hi[j]));
          lo[j] = pack_half2(a - hf.x, e - hf.y);
        }
        const uint32_t q_tm = *tmem_slot + lanes + 16 * g;
        tc::st16(q_tm + C::TM_QHI, hi);
        tc::st16(q_tm + C::TM_QLO, lo);
        tc::wait_st();
      }
    }
  }
  tc::fence_before();
  __syncthreads();  // the queries are in TMEM
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](int i, int parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar + i, parity & 1, CQ_NAP));
  };
  bool ok = true;

  if (warp == CQ_COPY_WARP) {
    // ======================= raw page copies =======================
    // lane c of the first eight has chunk c of each tile, and looks up its table
    // entry one tile before it is copied
    const int32_t* tbl = P.table + (size_t)(P.headwise ? b * Hkv + h : b) * P.max_blocks;
    const int bs_log2 = __ffs(bs) - 1;
    auto lookup = [&](int v) -> int {
      const int key = (v0 + v) * CQ_KT + 16 * lane;
      return lane < CQ_KT / 16 && v < nv && key < L ? __ldg(tbl + (key >> bs_log2)) : -1;
    };
    int entry = lookup(0), err = 0, v = 0, issued[2] = {0, 0};  // tiles whose K, and V, was copied
#pragma unroll 1
    for (; v < nv + 1 && ok; ++v) {
      const int st = v & 1;
      long long off = -1;
      if (v < nv) {  // tile v's place in the pages
        const int key = (v0 + v) * CQ_KT + 16 * lane;
        if (entry >= P.num_blocks) err |= DEVERR_BLOCK_RANGE;
        else if (entry >= 0) off = (((long long)entry * Hkv + h) * bs + (key & (bs - 1))) * C::R;
        if (off >= 0 && !KVQ_IN_BOUNDS(off + C::CHUNK <= (long long)P.num_blocks * Hkv * bs * C::R, P.dev_error)) off = -1;
        entry = lookup(v + 1);
      }
      const unsigned found = __ballot_sync(0xffffffffu, off >= 0);
      auto copy = [&](int i) -> bool {  // of K, or of V
        if (!wait((i ? QB_RAWVEMPTY : QB_RAWKEMPTY) + st, (v >> 1) ^ 1) || __any_sync(0xffffffffu, *abort_flag != 0)) return false;
        uint64_t* full = bar + (i ? QB_RAWVFULL : QB_RAWKFULL) + st;
        if (lane == 0) {
          if (i == 0) mask[v & 7] = (int)found;
          mbar_arrive_expect_tx(full, (uint32_t)(__popc(found) * C::CHUNK));
        }
        __syncwarp();
        issued[i] = v + 1;
        if (off >= 0)
          bulk_g2s(sm + C::OFF_RAW + (2 * st + i) * C::RAW + lane * C::CHUNK, (i ? P.v_pages : P.k_pages) + off, C::CHUNK, full);
        return true;
      };
      if (v < nv && !copy(0)) {
        ok = false;
        break;
      }
      // K's copy comes before the scales and V's after: V's waits for the P.V of tile v - 4, and S(v - 1) for the scales
      if constexpr (SCALES) {
        const int u = v - 1, su = u & 1;
        if (u >= 0) {  // scale and value of code 0 of tile u's keys; 0 for keys without data, which so add zeros
          // (tile u - 4 has left the place: S(u - 2), whose end is waited for, came after its P.V)
          if (!wait(QB_RAWKFULL + su, u >> 1) || !wait(QB_RAWVFULL + su, u >> 1) || !wait(QB_KEMPTY + su, (u >> 1) ^ 1)) {
            ok = false;
            break;
          }
          const uint8_t* rk = sm + C::OFF_RAW + su * 2 * C::RAW + C::DATA;
          const int chunks = mask[u & 7], left = L - (v0 + u) * CQ_KT;
          float* sc = reinterpret_cast<float*>(sm + C::OFF_SC) + (u & 3) * 5 * CQ_KT;
          uint32_t pads[2][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = 32 * i + lane;
            const bool has = ((chunks >> (j >> 4)) & 1) && j < left;
            pads[0][i] = has ? lds32(rk + j * C::R) : 0u;
            pads[1][i] = has ? lds32(rk + C::RAW + j * C::R) : 0u;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float ks, kz, vs, vz;  // (a pad of zeros: both are 0)
            pad_scale_zero<MODE>(pads[0][i], P.stego != 0, ks, kz);
            pad_scale_zero<MODE>(pads[1][i], P.stego != 0, vs, vz);
            if (ZEROS && (lane & 1)) vz -= vs;  // (odd keys' codes are one larger)
            sc[32 * i + lane] = ks;
            sc[CQ_KT + 32 * i + lane] = kz;
            sc[2 * CQ_KT + 32 * i + lane] = vs;
            sc[3 * CQ_KT + 32 * i + lane] = vz;
            // (not far below the zero point's, whose product with p is summed in fp32, and
            // not below -90: p, of values however small, stays below 2^104)
            const int es = (__float_as_uint(vs) >> 23) & 255, ez = ZEROS ? (int)((__float_as_uint(vz) >> 23) & 255) - 12 : 0;
            sc[4 * CQ_KT + 32 * i + lane] = (float)max(max(es, ez) - 126, -90);
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar + QB_KFULL + su);
        }
      }
      if (v < nv) ok = copy(1);
    }
    // the copies in flight land before the CTA ends, whoever gave up (there is nothing to wait for otherwise)
    for (int u = max(issued[0] - 2, 0); u < issued[0]; ++u) (void)wait(QB_RAWKFULL + (u & 1), u >> 1);
    for (int u = max(issued[1] - 2, 0); u < issued[1]; ++u) (void)wait(QB_RAWVFULL + (u & 1), u >> 1);
    err = __reduce_or_sync(0xffffffffu, err);
    if (err && lane == 0) flag_error(P.dev_error, err);
  } else if (warp >= CQ_PROD_WARP && warp < CQ_PROD_WARP + CQ_PRODUCERS) {
    // ======================= expansion =======================
    const int pt = tid - 32 * CQ_PROD_WARP;
    constexpr int PER = D / 8, STEP = 32 * CQ_PRODUCERS / PER;  // pieces of 8 dims per row; rows per pass of the threads
    const int c8 = pt % PER, row0 = pt / PER;
    // stores of rows row0 + STEP j: the swizzle takes 8 / STEP forms
    static_assert(STEP % 2 == 0, "a thread's rows are all even or all odd");
    constexpr int FORMS = STEP < 8 ? 8 / STEP : 1;
    int at[FORMS];
#pragma unroll
    for (int j = 0; j < FORMS; ++j) at[j] = (c8 >> 3) * C::HALF + tc::sw128_off(row0 + STEP * j, c8 & 7) - STEP * j * 128;
    auto expand = [&](const uint8_t* raw, uint8_t* tile, bool is_v, int v) {
      constexpr int U = 8;  // pieces in flight
      const uint32_t one = is_v ? row0 & 1 : 0;
      const int chunks = mask[v & 7], left = L - (v0 + v) * CQ_KT;
#pragma unroll 1
      for (int j0 = 0; j0 < CQ_KT / STEP; j0 += U) {
        uint4 x[U];
#pragma unroll
        for (int j = 0; j < U; ++j) x[j] = codes8<MODE>(raw + row0 * C::R + STEP * (j0 + j) * C::R, c8, one);
#pragma unroll
        for (int j = 0; j < U; ++j) {
          if (MODE == MODE_F8T && is_v) {  // rows without data may hold NaN codes, which a weight 0 does not cancel
            const int row = row0 + STEP * (j0 + j);
            if (row >= left || !((chunks >> (row >> 4)) & 1)) x[j] = make_uint4(0u, 0u, 0u, 0u);
          }
          *reinterpret_cast<uint4*>(tile + at[j % FORMS] + STEP * (j0 + j) * 128) = x[j];
        }
      }
    };
    // K runs a tile ahead of V, whose place is free only after the P.V before it:
    // K 0, K 1, V 0, K 2, V 1, ...
#pragma unroll 1
    for (int i = 0; i < 2 * nv; ++i) {
      const bool is_v = i == 2 * nv - 1 || (i > 0 && (i & 1) == 0);
      const int v = is_v ? (i == 2 * nv - 1 ? nv - 1 : (i >> 1) - 1) : (i + 1) >> 1, st = v & 1;
      if (!wait((is_v ? QB_RAWVFULL : QB_RAWKFULL) + st, v >> 1) || !wait((is_v ? QB_VEMPTY : QB_KEMPTY) + st, (v >> 1) ^ 1) ||
          __any_sync(0xffffffffu, *abort_flag != 0)) {
        ok = false;
        break;
      }
      expand(sm + C::OFF_RAW + (2 * st + (is_v ? 1 : 0)) * C::RAW, sm + (is_v ? C::OFF_V : C::OFF_K) + st * C::TILE, is_v, v);
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(bar + (is_v ? QB_VFULL : QB_KFULL) + st);
        tc::mbar_arrive(bar + (is_v ? QB_RAWVEMPTY : QB_RAWKEMPTY) + st);
      }
    }
  } else if (warp == CQ_MMA_WARP) {
    // ======================= MMA issue =======================
    const uint32_t one = tc::elect_one();
    const uint32_t id_s = idesc_f16_mn(CQ_ROWS, CQ_KT, false), id_o = idesc_f16_mn(CQ_ROWS, D, true);
    const uint64_t k_desc = tc::sw128_desc(smem_addr(sm + C::OFF_K)), v_desc = tc::mn_desc(smem_addr(sm + C::OFF_V), C::HALF);
    auto logits = [&](int u) {  // of the tile in stage u, to place u
      // the low terms first, while the sums that each step truncates are small
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint64_t bd = k_desc + (uint64_t)((u * C::TILE + (s >> 2) * C::HALF + (s & 3) * 32) >> 4);
          tc::mma_ts_if(one, tmem + u * CQ_KT, tmem + (i ? C::TM_QHI : C::TM_QLO) + 8 * s, bd, id_s, s > 0 || i > 0 ? 1u : 0u);
        }
      tc::commit_if(one, bar + QB_SFULL + u);
      tc::commit_if(one, bar + QB_KEMPTY + u);
    };
#pragma unroll 1
    for (int v = 0; v < min(nv, 2) && ok; ++v) {
      ok = wait(QB_KFULL + v, 0);
      tc::fence_after();
      if (ok) logits(v);
    }
#pragma unroll 1
    for (int v = 0; v < nv && ok; ++v) {
      const int u = v & 1;
      ok = wait(QB_VFULL + u, v >> 1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ok = ok && wait(QB_PFULL + 2 * u + i, v >> 1);
        if (!ok) break;
        tc::fence_after();
#pragma unroll
        for (int kk = 4 * i; kk < 4 * i + 4; ++kk) {
          const uint64_t bd = v_desc + (uint64_t)((u * C::TILE + kk * 16 * 128) >> 4);
          const uint32_t p_tm = tmem + u * CQ_KT + i * (CQ_KT / 2) + 8 * (kk & 3);
          tc::mma_ts_if(one, tmem + C::TM_O, p_tm, bd, id_o, v % CQ_FLUSH > 0 || kk > 0 ? 1u : 0u);
          tc::mma_ts_if(one, tmem + C::TM_O, p_tm + CQ_KT / 4, bd, id_o, 1u);
        }
        tc::commit_if(one, bar + QB_PVDONE + 2 * u + i);
      }
      if (!ok) break;
      tc::commit_if(one, bar + QB_VEMPTY + u);
      if (v + 2 < nv) {
        ok = wait(QB_KFULL + u, (v + 2) >> 1);
        tc::fence_after();
        if (ok) logits(u);
      }
      ok = ok && !__any_sync(0xffffffffu, *abort_flag != 0);
    }
    tc::commit_if(one, bar + QB_ODONE);
    tc::commit_if(one, bar + QB_DRAIN);  // every MMA issued by this warp has completed
    (void)wait(QB_DRAIN, 0);
  } else {
    // ======================= softmax =======================
    const uint32_t o_tm = tmem + lanes + C::TM_O;
    volatile float* pub = reinterpret_cast<volatile float*>(sm + C::OFF_M);
    const int qi = q0 + r / G;
    // where the rows end up: their outputs (rotated and unscaled until the end), or this part's record
    float* base = P.out;
    long long to = ((long long)(cq0 + qi) * Hq + h * G + r % G) * D;
    if (P.splits > 1) {
      base = P.part + ((((long long)b * Hkv + h) * (gridDim.x / P.splits) + qtile) * P.splits + sp) * split_record_floats(D);
      to = r * D;
    }
    if (!real) to = -1;
    float mine = -CUDART_INF_F, l = 0.0f, pz = 0.0f;  // of this group's keys, for the reference `mine`
    float held = -CUDART_INF_F;                       // group 0: the reference of what the rows hold
    float m = -CUDART_INF_F;
    const int u = g >> 1, half = g & 1;
#pragma unroll 1
    for (int t = g; t < 2 * nv; t += CQ_GROUPS) {  // half t & 1 of tile t / 2
      const int v = t >> 1;
      const uint32_t s_tm = tmem + lanes + g * CQ_HALF;
      if (!wait(QB_SFULL + u, v >> 1)) {
        ok = false;
        break;
      }
      tc::fence_after();
      const bool anew = half == 0 && v % CQ_FLUSH == 0;
      if (anew && v > 0) {  // (group 0) O so far is added to the rows
        if (!wait(QB_PUB + 4 * (CQ_GROUPS - 1) + quad, (t - 1) >> 2) || !wait(QB_PVDONE + ((t - 1) & 3), (t - 1) >> 2)) {
          ok = false;
          break;
        }
        tc::fence_after();
        m = pub[(CQ_GROUPS - 1) * CQ_ROWS + r];
        const float f = held == -CUDART_INF_F ? 0.0f : ex2(held - m);
        const bool more = v > CQ_FLUSH, add = more && __all_sync(0xffffffffu, f == 1.0f);
        // (a thread its own row: few instructions, and they are fetched anew each time)
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tc::ld32(o_tm + c, o);
          float4* p = reinterpret_cast<float4*>(base + to + c);
          float4 e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = more && !add && to >= 0 ? __ldcg(p + j) : make_float4(0.f, 0.f, 0.f, 0.f);
          tc::wait_ld();
          tc::regs_after_wait(o);
          if (to >= 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 x = make_float4(fmaf(e[j].x, f, __uint_as_float(o[4 * j])), fmaf(e[j].y, f, __uint_as_float(o[4 * j + 1])),
                                           fmaf(e[j].z, f, __uint_as_float(o[4 * j + 2])), fmaf(e[j].w, f, __uint_as_float(o[4 * j + 3])));
              if (add) tc::red_add4(reinterpret_cast<float*>(p + j), x);
              else __stcg(p + j, x);
            }
          }
        }
        tc::fence_before();
        held = m;
      }
      uint32_t y[CQ_HALF];
      tc::ld32(s_tm, y);
      tc::ld32(s_tm + 32, y + 32);
      const int left = L - (v0 + v) * CQ_KT - half * CQ_HALF, chunks = (mask[v & 7] >> (4 * half)) & 15;
      const float4* s4 = reinterpret_cast<const float4*>(sm + C::OFF_SC) + (v & 3) * (5 * CQ_KT / 4) + half * (CQ_HALF / 4);  // ks, kz, vs, vz, exponents: 32 apart
      tc::wait_ld();
      tc::regs_after_wait(y);
      float top[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
      const uint64_t rho2 = tc::pair32(rho, rho);
#pragma unroll
      for (int j = 0; j < CQ_HALF; j += 4) {  // s c.q'' + rho z, in units of beta
        if constexpr (SCALES) {
          const float4 ks = s4[j / 4];
          uint64_t z01 = 0, z23 = 0;
          if constexpr (ZEROS) {
            const float4 kz = s4[32 + j / 4];
            z01 = tc::fma_pair(tc::pair32(kz.x, kz.y), rho2, 0);
            z23 = tc::fma_pair(tc::pair32(kz.z, kz.w), rho2, 0);
          }
          const float2 a = tc::unpair32(tc::fma_pair(tc::pair32(ks.x, ks.y), tc::pair32(__uint_as_float(y[j]), __uint_as_float(y[j + 1])), z01));
          const float2 c = tc::unpair32(tc::fma_pair(tc::pair32(ks.z, ks.w), tc::pair32(__uint_as_float(y[j + 2]), __uint_as_float(y[j + 3])), z23));
          y[j] = __float_as_uint(a.x);
          y[j + 1] = __float_as_uint(a.y);
          y[j + 2] = __float_as_uint(c.x);
          y[j + 3] = __float_as_uint(c.y);
        }
      }
      if (left < CQ_HALF || chunks != 15) {  // (uniform over the CTA)
#pragma unroll
        for (int j = 0; j < CQ_HALF; ++j)
          if (j >= left || !((chunks >> (j / 16)) & 1)) y[j] = __float_as_uint(-CUDART_INF_F);
      }
      const uint64_t rb2 = tc::pair32(rb, rb);
      // the largest p s, as a power of two
#pragma unroll
      for (int j = 0; j < CQ_HALF; j += 8) {
        float t[8];
        if constexpr (SCALES) {
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            const float4 ex = s4[128 + (j + i) / 4];
            const float2 a = tc::unpair32(tc::fma_pair(tc::pair32(__uint_as_float(y[j + i]), __uint_as_float(y[j + i + 1])), rb2, tc::pair32(ex.x, ex.y)));
            const float2 c = tc::unpair32(tc::fma_pair(tc::pair32(__uint_as_float(y[j + i + 2]), __uint_as_float(y[j + i + 3])), rb2, tc::pair32(ex.z, ex.w)));
            t[i] = a.x; t[i + 1] = a.y; t[i + 2] = c.x; t[i + 3] = c.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] = __uint_as_float(y[j + i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = fmaxf(fmaxf(top[i], t[i]), t[4 + i]);
      }
      const float tmax = (SCALES ? 1.0f : rb) * fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) - CQ_BASE;
      if (t > 0) {  // the reference so far, from the group before
        if (!wait(QB_PUB + 4 * ((g - 1) & 3) + quad, (t - 1) >> 2)) {
          ok = false;
          break;
        }
        m = pub[((g - 1) & 3) * CQ_ROWS + r];
      }
      const bool grow = tmax > m + CQ_SLACK;
      const float m0 = m;
      m = grow ? tmax : m;
      pub[g * CQ_ROWS + r] = m;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar + QB_PUB + 4 * g + quad);
      if (!anew && __any_sync(0xffffffffu, grow && m0 != -CUDART_INF_F)) {
        if (!wait(QB_PVDONE + ((t - 1) & 3), (t - 1) >> 2)) {
          ok = false;
          break;
        }
        tc::fence_after();
        const float f = m0 == -CUDART_INF_F ? 1.0f : ex2(m0 - m);
#pragma unroll 1
        for (int c = 0; c < D; c += 8) {
          uint32_t o[8];
          tc::ld8(o_tm + c, o);
          tc::wait_ld();
          tc::regs_after_wait(o);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
          tc::st8(o_tm + c, o);
        }
        tc::wait_st();
        tc::fence_before();
      }
      const float ref = m == -CUDART_INF_F ? 0.0f : m;
      if (m != mine) {
        const float f = mine == -CUDART_INF_F ? 0.0f : ex2(mine - ref);
        l *= f;
        pz *= f;
        mine = m;
      }
      const uint64_t nref2 = tc::pair32(-ref, -ref);
      uint64_t sum[2] = {0, 0}, zsum[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < CQ_HALF; c += 32) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          float4 vs, vz;
          if constexpr (SCALES) vs = s4[64 + (c + 2 * j) / 4];
          if constexpr (ZEROS) vz = s4[96 + (c + 2 * j) / 4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int e = c + 2 * j + 2 * i;
            const float2 x = tc::unpair32(tc::fma_pair(tc::pair32(__uint_as_float(y[e]), __uint_as_float(y[e + 1])), rb2, nref2));
            uint64_t pp = tc::pair32(ex2(x.x), ex2(x.y));
            sum[i] = tc::add_pair(sum[i], pp);
            if constexpr (ZEROS) zsum[i] = tc::fma_pair(pp, i ? tc::pair32(vz.z, vz.w) : tc::pair32(vz.x, vz.y), zsum[i]);
            if constexpr (SCALES) pp = tc::mul_pair(pp, i ? tc::pair32(vs.z, vs.w) : tc::pair32(vs.x, vs.y));
            const float2 p = tc::unpair32(pp);
            // the high term cut to fp16's bits, so that the low one is the exact rest
            const float h0 = __uint_as_float(__float_as_uint(p.x) & 0xFFFFE000u), h1 = __uint_as_float(__float_as_uint(p.y) & 0xFFFFE000u);
            hi[j + i] = pack_half2(h0, h1);
            lo[j + i] = pack_half2(p.x - h0, p.y - h1);
          }
        }
        tc::st16(s_tm + c / 2, hi);
        tc::st16(s_tm + CQ_HALF / 2 + c / 2, lo);
      }
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar + QB_PFULL + g);
      const float2 a = tc::unpair32(tc::add_pair(sum[0], sum[1])), z = tc::unpair32(tc::add_pair(zsum[0], zsum[1]));
      l += a.x + a.y;
      pz += z.x + z.y;
      if (__any_sync(0xffffffffu, *abort_flag != 0)) {
        ok = false;
        break;
      }
    }
    // ---- the rows out.  The groups' sums meet, each for the last reference; a
    // thread makes 32 dims of a row, as at the start: from what was added up before,
    // O and the zero points' part, by the inverse RHT (or the INT8 V channel scales)
    // and 1 / l, or the part's record as it is.  (A warp to a row: 10 us of a CTA's end.)
    if (ok && nv > 0) ok = wait(QB_ODONE, 0);
    float* sums = reinterpret_cast<float*>(sm + C::OFF_SUM);
    int met = 0;
    auto meet = [&]() -> bool {  // the groups' warps that have these rows
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar + QB_MEET + quad);
      return wait(QB_MEET + quad, met++);
    };
    if (ok) {  // (the place is free when every P.V is done)
      sums[(3 * g + 0) * CQ_ROWS + r] = mine;
      sums[(3 * g + 1) * CQ_ROWS + r] = l;
      sums[(3 * g + 2) * CQ_ROWS + r] = pz;
      if (g == 0) sums[3 * CQ_GROUPS * CQ_ROWS + r] = held;
    } else {
      *abort_flag = 1;
    }
    ok = meet() && ok;
    ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
    if (ok) {
      tc::fence_after();
      const float hm = sums[3 * CQ_GROUPS * CQ_ROWS + r];
      float mt = -CUDART_INF_F, lt = 0.0f, pzt = 0.0f;
#pragma unroll
      for (int k = 0; k < CQ_GROUPS; ++k) mt = fmaxf(mt, sums[3 * k * CQ_ROWS + r]);
#pragma unroll
      for (int k = 0; k < CQ_GROUPS; ++k) {
        const float mk = sums[3 * k * CQ_ROWS + r], f = mk == -CUDART_INF_F ? 0.0f : ex2(mk - mt);
        lt = fmaf(f, sums[(3 * k + 1) * CQ_ROWS + r], lt);
        pzt = fmaf(f, sums[(3 * k + 2) * CQ_ROWS + r], pzt);
      }
      const float fh = hm == -CUDART_INF_F ? 0.0f : ex2(hm - mt);
      const bool part = P.splits > 1, both = rht && !part;
      float x[32];
      uint8_t* row = sm + C::OFF_K + r * (D * 4);  // whole rows (K and V are done with), 16-byte pieces XOR-swizzled by row
      float4* at = reinterpret_cast<float4*>(base + to + 32 * g);
      if (g < C::PIECES) {
        uint32_t o[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = 0;
        if (nv > 0) tc::ld32(o_tm + 32 * g, o);
        float4 e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = nv > CQ_FLUSH && to >= 0 ? __ldcg(at + j) : make_float4(0.f, 0.f, 0.f, 0.f);
        tc::wait_ld();
        tc::regs_after_wait(o);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[4 * j] = fmaf(e[j].x, fh, __uint_as_float(o[4 * j]) + pzt);
          x[4 * j + 1] = fmaf(e[j].y, fh, __uint_as_float(o[4 * j + 1]) + pzt);
          x[4 * j + 2] = fmaf(e[j].z, fh, __uint_as_float(o[4 * j + 2]) + pzt);
          x[4 * j + 3] = fmaf(e[j].w, fh, __uint_as_float(o[4 * j + 3]) + pzt);
        }
        if (both) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4*>(row + (((8 * g + j) ^ (r & 7)) << 4)) = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        }
      }
      if (both) {
        ok = meet();
        if (g < C::PIECES) {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = 0.0f;
#pragma unroll 1
          for (int k = 0; k < C::PIECES; ++k) {
            const float sg = __popc(g & k) & 1 ? -1.0f : 1.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 e = *reinterpret_cast<const float4*>(row + (((8 * k + j) ^ (r & 7)) << 4));
              x[4 * j] = fmaf(sg, e.x, x[4 * j]);
              x[4 * j + 1] = fmaf(sg, e.y, x[4 * j + 1]);
              x[4 * j + 2] = fmaf(sg, e.z, x[4 * j + 2]);
              x[4 * j + 3] = fmaf(sg, e.w, x[4 * j + 3]);
            }
          }
          wht_regs<32>(x);
        }
      }
      const float inv = lt > 0.0f ? 1.0f / lt : (lt == 0.0f ? 0.0f : lt);  // (a NaN stays one)
      if (part && g == 0 && to >= 0) reinterpret_cast<float2*>(base + CQ_ROWS * D)[r] = make_float2(mt, lt);
      if (g < C::PIECES && ok && to >= 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float4 f = *reinterpret_cast<const float4*>(ofac + 32 * g + 4 * j);
          f = part ? make_float4(1.0f, 1.0f, 1.0f, 1.0f) : make_float4(f.x * inv, f.y * inv, f.z * inv, f.w * inv);
          at[j] = make_float4(x[4 * j] * f.x, x[4 * j + 1] * f.y, x[4 * j + 2] * f.z, x[4 * j + 3] * f.w);
        }
      }
    }
  }
  if (!ok) {
    *abort_flag = 1;
    if (lane == 0) flag_error(P.dev_error, DEVERR_TIMEOUT);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == CQ_MMA_WARP) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

template <int MODE, int D>
static cudaError_t launch_crossq_t(const AttnParams& P, cudaStream_t stream) {
  using C = CqCfg<MODE, D>;
  static bool attr_set[64] = {false};  // once per device, not inside later calls, which may be captured
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(crossq_kernel<MODE, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int qtiles = (int)prefill_grid_x(P.max_q_per_seq, P.group);
  const dim3 grid((unsigned)qtiles * P.splits, P.num_kv_heads, P.batch);
  crossq_kernel<MODE, D><<<grid, CQ_THREADS, C::SMEM, stream>>>(P);
  if ((e = cudaGetLastError()) != cudaSuccess || P.splits == 1) return e;
  return launch_split_merge(P, qtiles, stream);
}

cudaError_t launch_crossq(const AttnParams& P, cudaStream_t stream) {
  switch (P.mode * 1000 + P.head_dim) {
    case MODE_INT4 * 1000 + 128: return launch_crossq_t<MODE_INT4, 128>(P, stream);
    case MODE_INT4 * 1000 + 64: return launch_crossq_t<MODE_INT4, 64>(P, stream);
    case MODE_INT2 * 1000 + 128: return launch_crossq_t<MODE_INT2, 128>(P, stream);
    case MODE_INT2 * 1000 + 64: return launch_crossq_t<MODE_INT2, 64>(P, stream);
    case MODE_INT8 * 1000 + 128: return launch_crossq_t<MODE_INT8, 128>(P, stream);
    case MODE_INT8 * 1000 + 64: return launch_crossq_t<MODE_INT8, 64>(P, stream);
    case MODE_I8T * 1000 + 128: return launch_crossq_t<MODE_I8T, 128>(P, stream);
    case MODE_I8T * 1000 + 64: return launch_crossq_t<MODE_I8T, 64>(P, stream);
    case MODE_F8T * 1000 + 128: return launch_crossq_t<MODE_F8T, 128>(P, stream);
    case MODE_F8T * 1000 + 64: return launch_crossq_t<MODE_F8T, 64>(P, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
