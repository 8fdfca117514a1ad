// kvq_cross16.cu -- cross attention over 16-bit (bf16) rows, dense or in pages,
// on the 5th-generation tensor cores (tcgen05, TMEM).
//
// For every query i of sequence b and q head: out = sum_j p_j v_j / sum_j p_j
// with p_j = exp(scale q_i . k_j) over all seq_lens[b] rows of the sequence,
// whatever the number of queries.  4 D flops per (query, q head, key).
//
// Design: one CTA of 12 warps per (up to 256 rows, kv head, sequence, part of
// the keys); a row is a (query, q head of the GQA group) pair, 128 rows make a
// tile, and the CTA's two tiles share every K and V tile of 128 keys.
//   warp 0          TMEM, and every tcgen05.mma: S = Q K^T (M = 128 rows, N = 128
//                   keys) and O += P V (N = D), the first half of the keys when
//                   its weights are there.  The oldest warp, since an SM's issue
//                   slots go to the oldest: as the youngest it was late by 300
//                   cycles at every step.
//   warps 1 and 2   tensor copies of K and of V (one warp for both held the next K
//                   back until a V stage was free): the rows land as they are,
//                   128-byte swizzled, ready to be operands: K as K-major, V as
//                   MN-major, so nothing is converted or transposed.
//   warps 4-7, 8-11 softmax of row tile 0 and 1, one thread per row: the row's
//                   128 logits from TMEM in one trip (a trip costs some 250
//                   cycles and 4 per column), their maximum, the weights, and
//                   those back to TMEM over the logits.  While one tile is in
//                   its softmax the tensor cores work on the other.  (Two threads
//                   per row, who must agree on the maximum: 8% slower.)
// A CTA with one row tile (few queries, fp32 ones) takes the other's logits' place
// for its next key tile: S(v + 1) is there when the softmax of v ends.
// bf16 x bf16 products are exact in the fp32 sums.  An fp32 query is three bf16
// terms (24 bits), three products into one sum, and one row tile per CTA.  The
// weights are two bf16 terms (17 bits: 2^-18 of a weight at most, 2e-6 of an
// output; one term alone would be 1e-3), so P.V takes twice its operations and
// the whole call 1.5 times 4 D per pair, which bounds it: two thirds of the
// tensor cores' rate.  The running maximum is a reference that moves, and O is
// rescaled, only when a logit passes it by 2^8.  The accumulators truncate, some
// 2^-25 of O per step of 16 keys and term (1.3e-5 of an output over 8192 keys):
// every CX_FLUSH tiles O is added in fp32 to the row where it will end up, and
// begins anew: 4e-6 to 6e-6.  (Every 8 tiles: half of that, 6% of the time.)
// Measured: 8 prompts of 1024 queries over 2048 .. 8192 rows (32 q and 8 kv heads
// of 128) 795 us in a loop of calls, 905 TFLOP/s of 4 D per pair and 1360 of the
// operations done (750 us alone, before the power cap lowers the clock); 5 queries
// over 131071 rows 62 us with the join, 4.3 TB/s.
// Rows that are not there (an evicted page, past the sequence's end): chunks of
// a page without an entry are copied from past the tensor's end, which gives
// zeros, and masked; value rows past the end of the sequence, which may hold
// anything, are zeroed in shared memory before the last P.V (a weight 0 does not
// cancel a NaN).
// Every wait is bounded; on a timeout the CTA reports KVQ_DEVERR_TIMEOUT,
// drains, frees its TMEM and returns.
//
// Sources: FastDeploy PR #7718 "Optimize AppendAttention for discrete head-wise
// block_idx" (head-wise tables, -1 sentinel); vllm-ascend-quantized-kv-cache
// METADATA, 运行机制 (gather, then dense attention).

#include <math_constants.h>

#include "kvq_cross.cuh"
#include "kvq_decode.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int CX_ROWS = PREFILL_ROWS;  // rows of a tile
constexpr int CX_KT = 128;             // keys of a tile
constexpr int CX_CHUNK = 16;           // rows of a page copied at a time
constexpr int CX_THREADS = 384;
constexpr int CX_MMA_WARP = 0, CX_COPY_WARP = 1;  // copies of K, and in the next warp of V
constexpr int CX_SOFTMAX_WARP = 4;                // the first of eight (warp 3 only loads queries)
constexpr int CX_FLUSH = 16;           // key tiles after which O is added up
constexpr float CX_SLACK = 8.0f;  // log2 units a logit may pass the reference maximum by
constexpr uint32_t CX_NAP = 20;   // ns between polls of a wait

template <int D, int TERMS>
struct CxCfg {
  static constexpr int TILES = TERMS == 1 ? 2 : 1;  // row tiles of a CTA
  static constexpr int HALF = CX_KT * 128;          // 64 dims of 128 rows: 128 lines of 128 bytes
  static constexpr int TILE = (D / 64) * HALF;      // 128 rows of Q, K or V
  static constexpr int NST = 2;                     // K stages, and V stages
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + TILES * TERMS * TILE;
  static constexpr int OFF_V = OFF_K + NST * TILE;
  static constexpr int OFF_MASK = OFF_V + NST * TILE;  // [4] chunks of tile v & 3 that hold rows
  // [TILES * 4 warps][32 rows][32 dims] fp32 on their way out; three-term queries leave no room for it
  static constexpr bool STAGED = TERMS == 1;
  static constexpr int OFF_OUT = OFF_MASK + 16;
  static constexpr int OFF_BAR = OFF_OUT + (STAGED ? TILES * 4 * tc::ADD_ROWS_BYTES : 0);
  static constexpr int NBAR = 18;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;  // TMEM address, abort flag
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  // TMEM columns: S (P over it: high terms, then low terms) and O of each row tile
  static constexpr int TM_O = 2 * CX_KT;
  static_assert(SMEM <= 232448, "shared memory");
};

// PFULL: of row tile (or, with one, key tile v & 1) t, the weights of half i of
// the keys, at 2 t + i; PVDONE: with one row tile, P.V of each key tile
enum { CB_KFULL = 0, CB_KEMPTY = 2, CB_VFULL = 4, CB_VEMPTY = 6, CB_SFULL = 8, CB_PFULL = 10, CB_ODONE = 14, CB_DRAIN = 15, CB_QFULL = 16,
       CB_PVDONE = 17 };

// kind::f16 with bf16 operands and fp32 sums; B K-major, or MN-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// 16 rows (TMEM lanes) x 64 columns: lane 4 i + j gets of columns 8 k + 2 j, + 1
// those of row i in r[4 k], r[4 k + 1] and of row i + 8 in r[4 k + 2], r[4 k + 3].
__device__ __forceinline__ void ld_rows16(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace

// Rows that sequence b's queries see, -1 where the sequence is skipped (its
// dense rows do not hold them).  `flag`: report what is wrong.
__device__ __forceinline__ int cross_keys(const AttnParams& P, int b, bool flag) {
  int L = load_input<false>(P.seq_lens + b);
  if (L < 0) {
    if (flag) flag_error(P.dev_error, DEVERR_SEQ_LEN);
    L = 0;
  }
  if (P.cu_kv) {
    const int c0 = load_input<false>(P.cu_kv + b), rows = load_input<false>(P.cu_kv + b + 1) - c0;
    if (rows < L || (L > 0 && (c0 < 0 || c0 > P.chunk_rows_total - L))) {
      if (flag) flag_error(P.dev_error, DEVERR_SEQ_LEN);
      return -1;
    }
  } else if (L > P.max_blocks * P.block_size) {
    if (flag) flag_error(P.dev_error, DEVERR_TABLE_RANGE);
    L = P.max_blocks * P.block_size;
  }
  return L;
}

template <int D, int TERMS>
__global__ void __launch_bounds__(CX_THREADS, 1) cross16_kernel(const __grid_constant__ AttnParams P) {
  using C = CxCfg<D, TERMS>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (P.splits > 1) allow_dependent_launch();  // the join of the parts may launch; it waits for this grid
  const int h = blockIdx.y;
  // barriers, TMEM and the sequence of this CTA, then (the copies already begin)
  // the queries
  volatile int* mask = reinterpret_cast<volatile int*>(sm + C::OFF_MASK);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 4);
  int* seq_slot = reinterpret_cast<int*>(sm + C::OFF_MISC + 8);
  if (warp == CX_COPY_WARP) {
    const int b0 = heavy_first_sequence(P, blockIdx.z);
    if (lane == 0) *seq_slot = b0;
  } else if (tid == 0) {
    for (int i = 0; i < C::NBAR; ++i)
      mbar_init(bar + i, i >= CB_PFULL && i < CB_PFULL + 4 ? CX_ROWS / 32 : i == CB_QFULL ? CX_THREADS - 63 : 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  __syncthreads();
  const int b = *seq_slot;
  const int sp = blockIdx.x % P.splits, block = blockIdx.x / P.splits;  // part of the keys, group of row tiles
  const int G = P.group, Hkv = P.num_kv_heads, QB = CX_ROWS / G;

  const int cq0 = __ldg(P.cu_q + b);
  int n = __ldg(P.cu_q + b + 1) - cq0;
  const bool first = tid == 0 && block == 0 && h == 0 && sp == 0;
  if (first && (n > P.max_q_per_seq || (n > 0 && (cq0 < 0 || cq0 > P.total_q - n)))) flag_error(P.dev_error, DEVERR_SEQ_LEN);
  n = min(n, P.max_q_per_seq);
  const int q0 = block * C::TILES * QB;
  if (q0 >= n || cq0 < 0) return;
  n = min(n, P.total_q - cq0);  // rows past the q that was given are neither read nor written
  if (q0 >= n) return;
  const int tiles = min(C::TILES, (n - q0 + QB - 1) / QB);
  const int L = cross_keys(P, b, first);
  if (L < 0) return;
  const int n_total = L / CX_KT + (L % CX_KT ? 1 : 0);  // (L may be next to 2^31)
  const int v0 = (int)((long long)sp * n_total / P.splits);
  const int nv = (int)((long long)(sp + 1) * n_total / P.splits) - v0;  // this part's key tiles

  uint32_t tmem = 0;
  bool started = true;
  if (warp == CX_COPY_WARP && lane == 0) {
    if (P.q_tma) {  // (queries of no row of this CTA come along, those past q as zeros: neither is stored)
      mbar_arrive_expect_tx(bar + CB_QFULL, (uint32_t)(tiles * (D / 64) * G * QB * 128));
      for (int t = 0; t < tiles; ++t)
#pragma unroll
        for (int hh = 0; hh < D / 64; ++hh)
          tc::tma_load_4d(sm + C::OFF_Q + t * C::TILE + hh * C::HALF, &P.q_map, 0, hh, h * G, cq0 + q0 + t * QB, bar + CB_QFULL);
    } else {
      tc::mbar_arrive(bar + CB_QFULL);
    }
  }
  const bool copies = warp == CX_COPY_WARP || warp == CX_COPY_WARP + 1;
  if (!copies) {
    if (warp == CX_MMA_WARP) tc::alloc(tmem_slot, 512);
    if (!P.q_tma) {
      // the rows' queries, as bf16 terms in the operand's layout: a warp per row (rows without a query: zeros)
      constexpr int EPL = D / 32, RU = 4, NW = CX_THREADS / 32 - 2;  // RU rows in flight
      const bool negative = P.softmax_scale < 0.0f;                  // carried by the queries
      const int d0 = lane * EPL, w0 = warp > CX_COPY_WARP ? warp - 2 : warp;
      for (int i0 = w0; i0 < tiles * CX_ROWS; i0 += RU * NW) {
        float x[RU][EPL];
#pragma unroll
        for (int u = 0; u < RU; ++u) {
          const int i = i0 + u * NW, r = i % CX_ROWS, qi = q0 + i / CX_ROWS * QB + r / G;
#pragma unroll
          for (int e = 0; e < EPL; ++e) x[u][e] = 0.0f;
          if (i < tiles * CX_ROWS && r / G < QB && qi < n && KVQ_IN_BOUNDS(cq0 + qi < P.total_q, P.dev_error))
            load_row_elems<EPL>(P.q, TERMS == 1 ? DT_BF16 : DT_F32, ((size_t)(cq0 + qi) * P.num_q_heads + h * G + r % G) * D + d0, x[u]);
        }
#pragma unroll
        for (int u = 0; u < RU; ++u) {
          const int i = i0 + u * NW, r = i % CX_ROWS, t = i / CX_ROWS;
          if (i < tiles * CX_ROWS) {
#pragma unroll
            for (int e = 0; e < EPL; ++e) x[u][e] = negative ? -x[u][e] : x[u][e];
#pragma unroll
            for (int k = 0; k < TERMS; ++k) {
              uint8_t* at = sm + C::OFF_Q + (t * TERMS + k) * C::TILE + (d0 >> 6) * C::HALF +
                            tc::sw128_off(r, (d0 & 63) >> 3) + 2 * (d0 & 7);
#pragma unroll
              for (int e = 0; e < EPL; e += 2) {
                const uint32_t w = pack_bf16x2(x[u][e], x[u][e + 1]);
                *reinterpret_cast<uint32_t*>(at + 2 * e) = w;
                x[u][e] -= __uint_as_float(w << 16);
                x[u][e + 1] -= __uint_as_float(w & 0xFFFF0000u);
              }
            }
          }
        }
      }
    }
    tc::fence_proxy_async();
    tc::fence_before();
    tc::mbar_arrive(bar + CB_QFULL);
    started = __all_sync(0xffffffffu, mbar_wait_bounded(bar + CB_QFULL, 0, CX_NAP));
    tc::fence_after();
    tmem = *tmem_slot;
    if (!started) *abort_flag = 1;
  }

  if (copies) {
    // ======================= copies =======================
    const int kv = warp - CX_COPY_WARP;
    // pages: lane c of the first eight has chunk c of each tile, and looks up its
    // table entry one tile before it is copied
    const bool paged = P.cu_kv == nullptr;
    const int32_t* tbl = P.table + (paged ? (size_t)(P.headwise ? b * Hkv + h : b) * P.max_blocks : 0);
    const int bs = P.block_size, bs_log2 = __ffs(bs) - 1;
    const int row0 = paged ? 0 : __ldg(P.cu_kv + b);
    auto lookup = [&](int v) -> int {
      const int key = (v0 + v) * CX_KT + CX_CHUNK * lane;
      return paged && lane < CX_KT / CX_CHUNK && v < nv && key < L ? __ldg(tbl + (key >> bs_log2)) : -1;
    };
    int entry = lookup(0), err = 0, issued = 0;  // tiles copied
    bool ok = true;
#pragma unroll 1
    for (int v = 0; v < nv && ok; ++v) {
      const int st = v & 1, parity = ((v >> 1) & 1) ^ 1;
      const int key0 = (v0 + v) * CX_KT;
      int row = P.chunk_rows_total;  // past the end: zeros
      if (entry >= P.num_blocks) err |= DEVERR_BLOCK_RANGE;
      else if (entry >= 0) row = (entry * Hkv + h) * bs + ((key0 + CX_CHUNK * lane) & (bs - 1));
      const unsigned found = paged ? __ballot_sync(0xffffffffu, row < P.chunk_rows_total) : 0xFFu;
      entry = lookup(v + 1);
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar + (kv ? CB_VEMPTY : CB_KEMPTY) + st, parity, CX_NAP)) ||
          __any_sync(0xffffffffu, *abort_flag != 0)) {
        ok = false;
        break;
      }
      uint64_t* full = bar + (kv ? CB_VFULL : CB_KFULL) + st;
      uint8_t* dst = sm + (kv ? C::OFF_V : C::OFF_K) + st * C::TILE;
      if (lane == 0) {
        if (kv == 0) mask[v & 3] = (int)found;
        mbar_arrive_expect_tx(full, C::TILE);
      }
      __syncwarp();
      issued = v + 1;
      if (paged) {
        if (lane < CX_KT / CX_CHUNK) {
#pragma unroll
          for (int hh = 0; hh < D / 64; ++hh)
            tc::tma_load_4d(dst + hh * C::HALF + lane * (CX_CHUNK * 128), &P.kv_map[kv], 0, hh, 0, row, full);
        }
      } else if (lane == 0) {
#pragma unroll
        for (int hh = 0; hh < D / 64; ++hh)
          tc::tma_load_4d(dst + hh * C::HALF, &P.kv_map[kv], 0, hh, h, row0 + key0, full);
      }
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) flag_error(P.dev_error, DEVERR_TIMEOUT);
    }
    // the copies in flight land before the CTA ends, whoever gave up (there is nothing to wait for otherwise)
    for (int u = max(issued - 2, 0); u < issued; ++u)
      (void)__all_sync(0xffffffffu, mbar_wait_bounded(bar + (kv ? CB_VFULL : CB_KFULL) + (u & 1), (u >> 1) & 1, CX_NAP));
    err = __reduce_or_sync(0xffffffffu, err);
    if (err && lane == 0) flag_error(P.dev_error, err);
  } else if (warp == CX_MMA_WARP) {
    // ======================= MMA issue =======================
    const uint32_t one = tc::elect_one();
    const uint32_t id_s = idesc_bf16(CX_ROWS, CX_KT, false), id_o = idesc_bf16(CX_ROWS, D, true);
    const uint64_t q_desc = tc::sw128_desc(smem_addr(sm + C::OFF_Q)), k_desc = tc::sw128_desc(smem_addr(sm + C::OFF_K));
    const uint64_t v_desc = tc::mn_desc(smem_addr(sm + C::OFF_V), C::HALF);  // (addresses are counted in 16 bytes)
    auto wait = [&](int i, int parity) -> bool { return __all_sync(0xffffffffu, mbar_wait_bounded(bar + i, parity & 1, CX_NAP)); };
    // S(t, v) goes where P(t, v - 1) was: P.V(t, v - 1) was issued before it, and
    // this thread's MMAs run in order; its commit tells the softmax of both.
    auto logits = [&](int t, int u, int st) {  // row tile t, to place u
      // the low terms first, while the sums that each step truncates are small
#pragma unroll
      for (int i = TERMS - 1; i >= 0; --i)
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const int at = ((s >> 2) * C::HALF + (s & 3) * 32) >> 4;
          tc::mma_ss_if(one, tmem + u * CX_KT, q_desc + (uint64_t)((t * TERMS + i) * (C::TILE >> 4) + at),
                        k_desc + (uint64_t)(st * (C::TILE >> 4) + at), id_s, s > 0 || i < TERMS - 1 ? 1u : 0u);
        }
      tc::commit_if(one, bar + CB_SFULL + u);
    };
    // O(t) += P V of key tile v, the weights at place u as they come
    auto values = [&](int t, int u, int v, int phase) -> bool {
      const uint32_t p = tmem + u * CX_KT, o = tmem + C::TM_O + t * D;
      const uint64_t vd = v_desc + (uint64_t)((v & 1) * (C::TILE >> 4));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!wait(CB_PFULL + 2 * u + i, phase)) return false;
        tc::fence_after();
#pragma unroll
        for (int kk = 4 * i; kk < 4 * i + 4; ++kk) {
          tc::mma_ts_if(one, o, p + 8 * kk, vd + kk * (16 * 128 >> 4), id_o, v % CX_FLUSH > 0 || kk > 0 ? 1u : 0u);
          tc::mma_ts_if(one, o, p + CX_KT / 2 + 8 * kk, vd + kk * (16 * 128 >> 4), id_o, 1u);
        }
      }
      return true;
    };
    bool ok = started;
    if (tiles == 1) {
#pragma unroll 1
      for (int v = 0; v < min(nv, 2) && ok; ++v) {
        ok = wait(CB_KFULL + v, 0);
        if (!ok) break;
        tc::fence_after();
        logits(0, v, v);
        tc::commit_if(one, bar + CB_KEMPTY + v);
      }
#pragma unroll 1
      for (int v = 0; v < nv && ok; ++v) {
        const int st = v & 1;
        ok = wait(CB_VFULL + st, v >> 1) && values(0, st, v, v >> 1);
        if (!ok) break;
        tc::commit_if(one, bar + CB_VEMPTY + st);
        tc::commit_if(one, bar + CB_PVDONE);
        if (v + 2 < nv) {
          ok = wait(CB_KFULL + st, (v + 2) >> 1);
          if (!ok) break;
          tc::fence_after();
          logits(0, st, st);
          tc::commit_if(one, bar + CB_KEMPTY + st);
        }
        ok = !__any_sync(0xffffffffu, *abort_flag != 0);
      }
    } else {
      if (ok && nv > 0 && (ok = wait(CB_KFULL, 0))) {
        tc::fence_after();
        logits(0, 0, 0);
        logits(1, 1, 0);
        tc::commit_if(one, bar + CB_KEMPTY);
      }
#pragma unroll 1
      for (int v = 0; v < nv && ok; ++v) {
        const int st = v & 1;
        const bool more = v + 1 < nv;
        ok = wait(CB_VFULL + st, v >> 1) && (!more || wait(CB_KFULL + (st ^ 1), (v + 1) >> 1));
#pragma unroll 1
        for (int t = 0; t < 2 && ok; ++t) {
          ok = values(t, t, v, v);
          if (ok && more) logits(t, t, st ^ 1);
        }
        if (!ok || __any_sync(0xffffffffu, *abort_flag != 0)) {
          ok = false;
          break;
        }
        tc::commit_if(one, bar + CB_VEMPTY + st);
        if (more) tc::commit_if(one, bar + CB_KEMPTY + (st ^ 1));
      }
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) flag_error(P.dev_error, DEVERR_TIMEOUT);
    }
    tc::commit_if(one, bar + CB_ODONE);
    tc::commit_if(one, bar + CB_DRAIN);  // every MMA issued by this warp has completed
    (void)wait(CB_DRAIN, 0);
  } else if (warp >= CX_SOFTMAX_WARP && warp / 4 - CX_SOFTMAX_WARP / 4 < tiles) {
    // ======================= softmax =======================
    const int t = warp / 4 - CX_SOFTMAX_WARP / 4, r = tid & (CX_ROWS - 1);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_tm = tmem + lanes + C::TM_O + t * D;
    const float sl = fmaxf(fabsf(P.softmax_scale) * 1.4426950408889634f, 1e-30f);
    // where the row ends up: its output, or this part's record
    const int qi = q0 + t * QB + r / G;
    const bool real = r / G < QB && qi < n && KVQ_IN_BOUNDS(cq0 + qi < P.total_q, P.dev_error);
    float* base = P.out;
    long long to = ((long long)(cq0 + qi) * P.num_q_heads + h * G + r % G) * D;  // from base
    if (P.splits > 1) {
      const long long tile = ((long long)b * Hkv + h) * (gridDim.x / P.splits * C::TILES) + block * C::TILES + t;
      base = P.part + (tile * P.splits + sp) * split_record_floats(D);
      to = r * D;
    }
    if (!real) to = -1;
    float m = -CUDART_INF_F, l = 0.0f;
    float held = -CUDART_INF_F;  // the reference of what `to` holds
    // The row at `to` = (itself 2^(held - m) + O) w; without `any` O is zeros,
    // without `more` the row is.
    auto add_up = [&](bool any, bool more, bool last, float w) {
      const float f = held == -CUDART_INF_F ? 0.0f : ex2(held - m);
      held = m;
      // O is added in memory, unread, while no reference of the warp's rows has moved
      const bool add = more && !last && __all_sync(0xffffffffu, f == 1.0f);
      if constexpr (C::STAGED) {
        tc::add_rows<D>(base, to, o_tm, f, w, any, more, add, sm + C::OFF_OUT + (t * 4 + (warp & 3)) * tc::ADD_ROWS_BYTES);
      } else {
        // in the layout of the 16-row loads: lane 4 i + j has dims 8 k + 2 j, + 1 of
        // rows i + 8 u, whole sectors
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = 8 * u + (lane >> 2);
          const long long at = __shfl_sync(0xffffffffu, to, row);
          const float g = __shfl_sync(0xffffffffu, f, row), x = __shfl_sync(0xffffffffu, w, row);
          float* p = base + at + 2 * (lane & 3);
#pragma unroll 1
          for (int c = 0; c < D; c += 64) {
            uint32_t o[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0;
            if (any) {
              ld_rows16(o_tm + ((uint32_t)(16 * (u >> 1)) << 16) + c, o);
              tc::wait_ld();
              tc::regs_after_wait(o);
            }
            if (at < 0) continue;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float o0 = __uint_as_float(o[4 * k + 2 * (u & 1)]), o1 = __uint_as_float(o[4 * k + 2 * (u & 1) + 1]);
              float2* to2 = reinterpret_cast<float2*>(p + c + 8 * k);
              const float2 e = more ? __ldcg(to2) : make_float2(0.0f, 0.0f);
              __stcg(to2, make_float2(fmaf(e.x, g, o0) * x, fmaf(e.y, g, o1) * x));
            }
          }
        }
      }
    };
    const uint64_t sl2 = tc::pair32(sl, sl), minus1 = tc::pair32(-1.0f, -1.0f);
    bool ok = started;
#pragma unroll 1
    for (int v = 0; v < nv; ++v) {
      // every decision around a .sync.aligned TMEM access is warp-uniform
      const int u = tiles == 1 ? v & 1 : t, phase = tiles == 1 ? v >> 1 : v;
      const uint32_t s_tm = tmem + lanes + u * CX_KT;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar + CB_SFULL + u, phase & 1, CX_NAP))) {
        ok = false;
        break;
      }
      tc::fence_after();
      // O may be touched when P.V(v - 1) is done: with two row tiles it is, since
      // S(v) was committed after it
      auto o_is_done = [&]() -> bool {
        if (tiles > 1 || v == 0) return true;
        const bool good = __all_sync(0xffffffffu, mbar_wait_bounded(bar + CB_PVDONE, (v - 1) & 1, CX_NAP));
        tc::fence_after();
        return good;
      };
      if (v > 0 && v % CX_FLUSH == 0) {
        if (!o_is_done()) {
          ok = false;
          break;
        }
        add_up(true, v > CX_FLUSH, false, 1.0f);
      }
      uint32_t y[CX_KT];
#pragma unroll
      for (int c = 0; c < CX_KT; c += 32) tc::ld32(s_tm + c, y + c);
      const int left = L - (v0 + v) * CX_KT;  // keys of the sequence from this tile on
      const int chunks = mask[v & 3];
      if (t == 0 && left < CX_KT && r >= left) {  // a value row past the end, before the P.V that would read it
        ok = mbar_wait_bounded(bar + CB_VFULL + (v & 1), (v >> 1) & 1, CX_NAP);
        uint8_t* row = sm + C::OFF_V + (v & 1) * C::TILE + r * 128;
        if (ok) {
#pragma unroll
          for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
            for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(row + hh * C::HALF + 16 * c) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async();
      }
      tc::wait_ld();
      tc::regs_after_wait(y);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      if (left < CX_KT || chunks != 0xFF) {  // (uniform over the CTA)
#pragma unroll
        for (int j = 0; j < CX_KT; ++j)
          if (j >= left || !((chunks >> (j / CX_CHUNK)) & 1)) y[j] = __float_as_uint(-CUDART_INF_F);
      }
      float top[4];  // four chains: one is 128 latencies long
#pragma unroll
      for (int j = 0; j < 4; ++j) top[j] = fmaxf(__uint_as_float(y[j]), __uint_as_float(y[j + 4]));
#pragma unroll
      for (int j = 8; j < CX_KT; j += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = fmaxf(fmaxf(top[i], __uint_as_float(y[j + i])), __uint_as_float(y[j + 4 + i]));
      const float tmax = sl * fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      const bool grow = tmax > m + CX_SLACK;
      const bool resc = grow && m != -CUDART_INF_F;
      if (__any_sync(0xffffffffu, resc)) {
        const float f = resc ? ex2(m - tmax) : 1.0f;
        if (v % CX_FLUSH > 0) {  // (else O begins anew)
          if (!o_is_done()) {
            ok = false;
            break;
          }
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
        }
        l *= f;
      }
      m = grow ? tmax : m;
      const float ref = m == -CUDART_INF_F ? 0.0f : m;
      const uint64_t nref2 = tc::pair32(-ref, -ref);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < CX_KT; c += 32) {  // 32 keys: 16 columns of high terms and 16 of low ones
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 x = tc::unpair32(tc::fma_pair(tc::pair32(__uint_as_float(y[c + 2 * j]), __uint_as_float(y[c + 2 * j + 1])), sl2, nref2));
          const float p0 = ex2(x.x), p1 = ex2(x.y);
          const uint64_t pp = tc::pair32(p0, p1);
          sum[j & 1] = tc::add_pair(sum[j & 1], pp);
          hi[j] = pack_bf16x2(p0, p1);
          const float2 d = tc::unpair32(
              tc::fma_pair(tc::pair32(__uint_as_float(hi[j] << 16), __uint_as_float(hi[j] & 0xFFFF0000u)), minus1, pp));
          lo[j] = pack_bf16x2(d.x, d.y);
        }
        tc::st16(s_tm + c / 2, hi);
        tc::st16(s_tm + CX_KT / 2 + c / 2, lo);
        if (c % 64 == 32) {  // a half of the keys: P.V may begin with it
          tc::wait_st();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar + CB_PFULL + 2 * u + c / 64);
        }
      }
      const float2 sum2 = tc::unpair32(tc::add_pair(sum[0], sum[1]));
      l += sum2.x + sum2.y;
      if (__any_sync(0xffffffffu, *abort_flag != 0)) {
        ok = false;
        break;
      }
    }
    // ---- the rows out: divided by the sum, or as this part's record
    if (ok && nv > 0 && !__all_sync(0xffffffffu, mbar_wait_bounded(bar + CB_ODONE, 0, CX_NAP))) ok = false;
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) flag_error(P.dev_error, DEVERR_TIMEOUT);
    } else {
      tc::fence_after();
      const bool part = P.splits > 1;
      if (part) reinterpret_cast<float2*>(base + CX_ROWS * D)[r] = make_float2(m, l);
      add_up(nv > 0, nv > CX_FLUSH, true, part ? 1.0f : l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l));  // (a NaN stays one)
    }
  }

  tc::fence_before();
  __syncthreads();
  if (warp == CX_MMA_WARP) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

// Joins the parts of one (query, q head) row: log-sum-exp weights, then the
// inverse RHT (or the INT8 V channel scales) and 1 / l.  W warps per row each
// take every W-th group of eight parts (their loads in flight together) and meet
// in shared memory: one row of five queries over 38 parts took 16.5 us with one
// warp and four loads at a time.  Lane l has dims l * EPL .. + EPL - 1.
template <int D, int W>
__global__ void __launch_bounds__(256) split_merge_kernel(const AttnParams P, int qtiles) {
  constexpr int EPL = D / 32, U = 8, ROWS = 8 / W;  // rows of a CTA
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % W, G = P.group, Hkv = P.num_kv_heads;
  const int QB = PREFILL_ROWS / G;
  const long long wid = (long long)blockIdx.x * ROWS + warp / W;
  const int row = (int)(wid % PREFILL_ROWS);
  const long long tile = wid / PREFILL_ROWS;  // (b * Hkv + h) * qtiles + qtile
  if (tile >= (long long)P.batch * Hkv * qtiles) return;  // (whole CTAs, for W > 1; so below)
  const int qtile = (int)(tile % qtiles), h = (int)(tile / qtiles % Hkv), b = (int)(tile / qtiles / Hkv);
  grid_dependency_wait();  // every record is written
  const int cq0 = load_input<false>(P.cu_q + b);
  const int n = min(load_input<false>(P.cu_q + b + 1) - cq0, P.max_q_per_seq);
  const int qi = qtile * QB + row / G;
  if (row / G >= QB || qi >= n || cq0 < 0 || cq0 + qi >= P.total_q) return;
  if (cross_keys(P, b, false) < 0) return;  // (a skipped sequence has no records)
  float m = -CUDART_INF_F, l = 0.0f, o[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) o[e] = 0.0f;
  const float* rec0 = P.part + tile * P.splits * split_record_floats(D);
  for (int s0 = U * part; s0 < P.splits; s0 += U * W) {
    float2 ml[U];
    float v[U][EPL];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float* rec = rec0 + min(s0 + u, P.splits - 1) * split_record_floats(D);
      ml[u] = __ldcg(reinterpret_cast<const float2*>(rec + PREFILL_ROWS * D) + row);
      if constexpr (EPL == 4) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(rec + row * D) + lane);
        v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
      } else {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(rec + row * D) + lane);
        v[u][0] = x.x; v[u][1] = x.y;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u >= P.splits || ml[u].y == 0.0f) continue;  // no visible key in this part
      const float mn = fmaxf(m, ml[u].x);
      const float f = m == -CUDART_INF_F ? 0.0f : ex2(m - mn), w = ex2(ml[u].x - mn);
      m = mn;
      l = l * f + ml[u].y * w;
#pragma unroll
      for (int e = 0; e < EPL; ++e) o[e] = o[e] * f + v[u][e] * w;
    }
  }
  if constexpr (W > 1) {
    __shared__ float sm_m[W], sm_l[W], sm_o[W][D];
    if (lane == 0) {
      sm_m[part] = m;
      sm_l[part] = l;
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) sm_o[part][EPL * lane + e] = o[e];
    __syncthreads();
    if (part != 0) return;
    const float m0 = m;
#pragma unroll
    for (int w = 1; w < W; ++w) m = fmaxf(m, sm_m[w]);
    const float f0 = m0 == -CUDART_INF_F ? 0.0f : ex2(m0 - m);
    l *= f0;
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] *= f0;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const float f = sm_m[w] == -CUDART_INF_F ? 0.0f : ex2(sm_m[w] - m);
      l = fmaf(f, sm_l[w], l);
#pragma unroll
      for (int e = 0; e < EPL; ++e) o[e] = fmaf(f, sm_o[w][EPL * lane + e], o[e]);
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);  // (a NaN stays one)
  if (P.mode == MODE_INT8) {
    const float* am = P.ch_amax + ((size_t)Hkv + h) * D + lane * EPL;
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] *= __fdiv_rn(am[e], 127.0f) * inv;
  } else if (P.signs) {
    wht_warp<EPL>(o, lane);
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] = (__ldg(P.signs + lane * EPL + e) < 0 ? -o[e] : o[e]) * (inv / (float)D);
  } else {
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] *= inv;
  }
  float* out = P.out + ((size_t)(cq0 + qi) * P.num_q_heads + h * G + row % G) * D + lane * EPL;
  if constexpr (EPL == 4) *reinterpret_cast<float4*>(out) = make_float4(o[0], o[1], o[2], o[3]);
  else *reinterpret_cast<float2*>(out) = make_float2(o[0], o[1]);
}

template <int D>
static cudaError_t launch_split_merge_d(const AttnParams& P, int qtiles, cudaStream_t stream) {
  const long long rows = (long long)P.batch * P.num_kv_heads * qtiles * PREFILL_ROWS;
  if (P.splits > 8)  // more parts than one warp has in flight
    return launch_dependent(split_merge_kernel<D, 8>, dim3((unsigned)rows), dim3(256), 0, stream, P, qtiles);
  return launch_dependent(split_merge_kernel<D, 1>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, stream, P, qtiles);
}
cudaError_t launch_split_merge(const AttnParams& P, int qtiles, cudaStream_t stream) {
  return P.head_dim == 128 ? launch_split_merge_d<128>(P, qtiles, stream) : launch_split_merge_d<64>(P, qtiles, stream);
}

template <int D, int TERMS>
static cudaError_t launch_cross16_t(const AttnParams& P, cudaStream_t stream) {
  using C = CxCfg<D, TERMS>;
  static bool attr_set[64] = {false};  // once per device, not inside later calls, which may be captured
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(cross16_kernel<D, TERMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int blocks = (int)cross16_blocks(P.max_q_per_seq, P.group, TERMS > 1);
  const dim3 grid((unsigned)blocks * P.splits, P.num_kv_heads, P.batch);
  cross16_kernel<D, TERMS><<<grid, CX_THREADS, C::SMEM, stream>>>(P);
  if ((e = cudaGetLastError()) != cudaSuccess || P.splits == 1) return e;
  return launch_split_merge(P, blocks * C::TILES, stream);
}

cudaError_t launch_cross16(const AttnParams& P, cudaStream_t stream) {
  const bool f32 = P.dtype == DT_F32;
  if (P.head_dim == 128) return f32 ? launch_cross16_t<128, 3>(P, stream) : launch_cross16_t<128, 1>(P, stream);
  return f32 ? launch_cross16_t<64, 3>(P, stream) : launch_cross16_t<64, 1>(P, stream);
}

}  // namespace kvq
