// kvq_decode16.cu -- split-KV decode attention over 16-bit (bf16) pages.
//
// For every sequence b and q head: out = sum_j p_j v_j / sum_j p_j with
// p_j = exp(scale q . k_j) over the visible keys j, K and V rows read as they
// lie in the pages (no codes, no scale, no rotation).  4 D G flops for the
// 4 D bytes of one key of one kv head (G q heads share it): bound by memory
// for every group the library takes.
//
// Design.  The unit of work is a chunk of 16 keys (every page holds whole
// chunks: 16 rows, contiguous).  The concatenated chunk lists of all
// (sequence, kv head) pairs are cut into one contiguous, equal slice per warp,
// whatever the context lengths; a warp writes one partial record (running
// maximum, sum, unnormalised output) each time its slice leaves a pair, and a
// second kernel joins the records of a pair.
//  * Chunk look-up is lane-parallel: lane i of a warp finds the pair, the page
//    and the 16-bit visibility mask of chunk x + i of the slice, 32 chunks at
//    a time and one such block ahead, so that the table's latency and the
//    change of pair cost the loop nothing.
//  * K and V go from global memory straight to the registers of the matrix
//    instructions (m16n8k16, bf16 x bf16 with fp32 sums): the order of the
//    dims of a dot product is free, so a lane reads 16 consecutive bytes of a
//    key row and these are its operand words for two k-steps; the order of the
//    output dims is free too, so a lane reads 16 bytes (8 dims) of four key
//    rows and eight byte permutes pair them by key.  No shared memory, no
//    wait: the loads of chunk x + 1 are in flight while chunk x is computed
//    (K's from the end of QK^T on, V's from the end of P.V on).
//  * QK^T has M = 16 keys and N = 8 q heads: exact products of bf16 inputs.
//    An fp32 q is split into three bf16 terms (24 bits), three instructions
//    into the same sums.  P.V has M = 16 dims, K = 16 keys, N = 8 heads; the
//    weights, an 8 x 8 transpose away (movmatrix), are split into three bf16
//    terms for the same reason: two terms would keep 16 bits, an error of
//    2e-6 of the output where the fp32 sums themselves are off by 1e-6.
//  * The maximum is a reference, not the exact one: it moves (and the sums and
//    outputs are rescaled) only when a logit passes it by 2^8, so most chunks
//    take one vote and no reduction.  Weights up to 2^8 lose nothing in fp32
//    or bf16, whose exponents have the range.
//    Sums of one chunk are joined to the running ones in fp32: carried in the
//    instructions' accumulators, which truncate, they were off by 3e-6 to 6e-6
//    of the output over slices of 64 to 160 chunks, now 4e-7.
//  * Masked keys: the logit is replaced by -inf and the value row by zeros,
//    since a stale slot may hold a NaN, which a zero weight would not cancel.
// Measured (one GB300, 6792 GB/s a plain copy's): 64 sequences of 1024 .. 8192
// keys, 8 kv heads, 1.21 GB: 182 us a call, 6.6 TB/s (with fp32 queries too; 21%
// of the issue slots, 18% of the tensor pipe busy); 32 sequences of
// 32768 with windows, 2.42 GB: 345 us, 7.0 TB/s; one sequence of 131071 keys,
// 4 kv heads: 50 us, 5.4 TB/s (its start and the merge of 1824 records are 10 us
// of it).  12 warps of 168 registers keep 96 KB per SM in flight; 13 and 14,
// which spill, take 229 and 235 us.  At D = 64 a warp has half as much in
// flight: 16 warps of 125 registers read 0.60 GB (the first case's lengths) in
// 99 us against 103 with 12 and 141 with 24, 8 sequences of 65536 in 164 against
// 174 us (6.5 TB/s).

#include <math_constants.h>

#include "kvq_decode.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int D16_KEYS = 16;       // keys per chunk
// Warps per CTA, one CTA per SM: as many as 64 K registers hold without spills.
__host__ __device__ constexpr int d16_warps(int head_dim) { return head_dim == 128 ? 12 : 16; }
constexpr int D16_RUNS = 2048;     // entries of the prefix sums over the pairs
constexpr int D16_MIN_CHUNKS = 1;  // per warp, at least
constexpr int D16_WIDE_MERGE = 16;  // records per pair from which a CTA joins one head
constexpr int D16_DIRECT_COST = 6;  // see launch_decode16_d
constexpr float D16_SLACK = 8.0f;  // log2 units a logit may pass the reference maximum by

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {  // read once: not kept in L1
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// D = A * B, m16n8k16, bf16 inputs, fp32 sums.
__device__ __forceinline__ void mma_bf16_fresh(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// D = A * B + D.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Three bf16 terms whose sum is (lo, hi) to 24 bits each: what is left after
// a rounding to 8 bits is exact in fp32, so the third term's rounding, 2^-24
// of the value at most, is all that is lost.
__device__ __forceinline__ void split3(float lo, float hi, uint32_t (&t)[3]) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    t[k] = pack_bf16(lo, hi);
    if (k < 2) {
      lo -= __uint_as_float(t[k] << 16);
      hi -= __uint_as_float(t[k] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 16 ? 0xFFFFu : (1u << n) - 1u); }

// What the loop needs of one chunk.
struct Chunk {
  int bh;         // (sequence, kv head) pair
  int row;        // chunk of 16 rows in the pool, -1: nothing to read
  uint32_t mask;  // bit k: key k is visible
};

// DIRECT: one CTA per pair instead, its warps' shares joined in shared memory
// and written out: no records, no prefix sums and no second launch, for calls
// of few and short sequences.
template <int D, bool Q32, bool DIRECT>
__global__ void __launch_bounds__(d16_warps(D) * 32, 1) decode16_kernel(const AttnParams P, const DecodeWs ws) {
  constexpr int WARPS = d16_warps(D), NT = WARPS * 32;
  constexpr int JK = D / 32;  // 16-byte pieces of a key row per lane
  constexpr int JV = D / 64;  // 16-byte pieces of a value row per lane
  constexpr int ROW = 2 * D;  // bytes
  // Q32: the q terms, [warp][3][JK][32 lanes][16 bytes]; DIRECT: then the
  // warps' outputs [warp][G][D], maxima and sums [warp][G]
  extern __shared__ __align__(16) uint8_t qsm[];
  __shared__ int run_start[DIRECT ? 1 : D16_RUNS + 1];
  __shared__ int wtot[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int G = P.group, Hkv = P.num_kv_heads, bs = P.block_size, BH = P.batch * Hkv;
  const int bs_log2 = __ffs(bs) - 1;
  // The kernel before may still run (programmatic launch).  The write of the
  // same call touches neither queries, tables and lengths nor the workspace,
  // so only the pages wait for it; another may be writing the former or
  // reading memory that has since become the latter.
  if (P.new_k == nullptr) grid_dependency_wait();
  int lo, hi, gw = 0, items = 1, nruns = 1;
  if constexpr (DIRECT) {
    const bool reports = threadIdx.x == 0 && blockIdx.x % Hkv == 0;
    const TileList t = tile_list<false>(P, blockIdx.x / Hkv, blockIdx.x % Hkv, reports, D16_KEYS);
    lo = slice_lo(warp, t.n_virt, WARPS);
    hi = slice_lo(warp + 1, t.n_virt, WARPS);
  } else {
    allow_dependent_launch();  // the merge kernel may launch; it waits for this grid to finish

    // Prefix sums of the pairs' chunk counts, over runs of `items` pairs; CTA 0
    // also publishes every pair's first chunk for the merge and reports bad lengths.
    items = (BH + D16_RUNS - 1) / D16_RUNS;
    nruns = (BH + items - 1) / items;
    const int rpt = (nruns + NT - 1) / NT;  // runs per thread
    {
      const int first = min(BH, (int)threadIdx.x * rpt * items), last = min(BH, first + rpt * items);
      int sum = 0;
      for (int bh = first; bh < last; ++bh) sum += tile_list<false>(P, bh / Hkv, bh % Hkv, false, D16_KEYS).n_virt;
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) wtot[warp] = incl;
      __syncthreads();
      int x = incl - sum;
      for (int w = 0; w < warp; ++w) x += wtot[w];
      for (int bh = first; bh < last; ++bh) {
        if (bh % items == 0) run_start[bh / items] = x;
        const int n = tile_list<false>(P, bh / Hkv, bh % Hkv, blockIdx.x == 0 && bh % Hkv == 0, D16_KEYS).n_virt;
        if (blockIdx.x == 0) ws.tile_start[bh] = x;
        x += n;
      }
      if (threadIdx.x == NT - 1) {
        run_start[nruns] = x;
        if (blockIdx.x == 0) ws.tile_start[BH] = x;
      }
      __syncthreads();
    }
    const int T = run_start[nruns];
    const int nw = stream_workers(T, gridDim.x * WARPS, ws.fixed_workers, D16_MIN_CHUNKS);
    gw = warp * gridDim.x + blockIdx.x;  // few slices: spread over the SMs
    if (gw >= nw) return;  // whole warp; no CTA-wide barrier follows
    lo = slice_lo(gw, T, nw);
    hi = slice_lo(gw + 1, T, nw);
    if (lo >= hi) return;
  }

  int err = 0;
  auto look_up = [&](int at) -> Chunk {  // of chunk `at` of the slice; lanes past its end get nothing
    Chunk r;
    r.bh = -1;
    r.row = -1;
    r.mask = 0;
    if (at >= hi - lo) return r;
    const int x = lo + at;
    int bh = blockIdx.x, start = 0;
    if constexpr (!DIRECT) {
      int a = 0, z = nruns;
      while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (run_start[mid] <= x) a = mid;
        else z = mid;
      }
      bh = a * items;
      start = run_start[a];
    }
    TileList t = tile_list<false>(P, bh / Hkv, bh % Hkv, false, D16_KEYS);
    if constexpr (!DIRECT) {
      while (start + t.n_virt <= x) {  // (items > 1 only)
        start += t.n_virt;
        ++bh;
        t = tile_list<false>(P, bh / Hkv, bh % Hkv, false, D16_KEYS);
      }
    }
    r.bh = bh;
    const int key = D16_KEYS * tile_of(t, x - start);
    r.mask = low_bits(t.Leff - key);
    if (t.W > 0) {
      const int before = t.L - t.W - key;  // keys of the chunk before the window
      r.mask &= ~low_bits(before) | low_bits(P.sink - key);
    }
    if (!KVQ_IN_BOUNDS((key >> bs_log2) < P.max_blocks, P.dev_error)) r.mask = 0;
    if (r.mask) {
      const int e = load_input<false>(P.table + (size_t)(P.headwise ? bh : bh / Hkv) * P.max_blocks + (key >> bs_log2));
      if (e >= P.num_blocks) err |= DEVERR_BLOCK_RANGE;
      else if (e >= 0) r.row = (e * Hkv + bh % Hkv) * (bs / D16_KEYS) + ((key & (bs - 1)) / D16_KEYS);
    }
    return r;
  };

  uint4 ka[JK], kb[JK], vr[4][JV];
  auto load_k = [&](int row) {
    if (row < 0) return;
    const uint8_t* p = P.k_pages + (size_t)row * (D16_KEYS * ROW) + g * ROW + c * 16;
#pragma unroll
    for (int j = 0; j < JK; ++j) {
      ka[j] = ld_stream(p + 64 * j);
      kb[j] = ld_stream(p + 8 * ROW + 64 * j);
    }
  };
  auto load_v = [&](int row) {
    if (row < 0) return;
    const uint8_t* p = P.v_pages + (size_t)row * (D16_KEYS * ROW) + 2 * c * ROW + g * 16;
#pragma unroll
    for (int j = 0; j < JV; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k)  // keys 2c, 2c+1, 2c+8, 2c+9
        vr[k][j] = ld_stream(p + (8 * (k >> 1) + (k & 1)) * ROW + 128 * j);
  };

  uint4 qf[Q32 ? 1 : JK];  // head g's dims 32 j + 8 c .. + 7
  uint8_t* qw = qsm + (size_t)warp * 3 * JK * 512 + lane * 16;
  float acc[JV][4][4];     // [.][w]: dims 64 j + 8 g + 2 w, + 1 of heads 2 c, 2 c + 1
  float m[2], l[2];
  const float sl = P.softmax_scale * 1.4426950408889634f;
  auto begin_pair = [&](int bh) {
    const size_t q0 = ((size_t)(bh / Hkv) * P.num_q_heads + (bh % Hkv) * G + g) * D + 8 * c;
#pragma unroll
    for (int j = 0; j < JK; ++j) {
      if constexpr (Q32) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.0f;
        if (g < G) load_row_elems<8, false>(P.q, DT_F32, q0 + 32 * j, x);
        uint32_t t[4][3];
#pragma unroll
        for (int i = 0; i < 4; ++i) split3(x[2 * i], x[2 * i + 1], t[i]);
#pragma unroll
        for (int k = 0; k < 3; ++k)
          *reinterpret_cast<uint4*>(qw + (k * JK + j) * 512) = make_uint4(t[0][k], t[1][k], t[2][k], t[3][k]);
      } else {
        qf[j] = g < G ? load_input<false>(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(P.q) + 2 * q0) + 4 * j)
                      : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < JV; ++j)
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][w][i] = 0.0f;
    m[0] = m[1] = -CUDART_INF_F;
    l[0] = l[1] = 0.0f;
  };
  float* osm = reinterpret_cast<float*>(qsm + (Q32 ? (size_t)WARPS * 3 * JK * 512 : 0));
  float2* mlsm = reinterpret_cast<float2*>(osm + (size_t)WARPS * G * D);
  // The record of (worker gw, pair bh), or the warp's share in shared memory.
  auto end_pair = [&](int bh) {
    const int rec = DIRECT ? warp : gw + bh;
    if (!DIRECT && !KVQ_IN_BOUNDS(rec < ws.n_partials, P.dev_error)) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
      const int head = 2 * c + i;
      if (head < G) {
        // (a NaN among the logits may have left no maximum: the join wants a finite one to add the NaN by)
        if (g == 0)
          (DIRECT ? mlsm : ws.part_ml)[(size_t)rec * G + head] = make_float2(isnan(l[i]) ? fmaxf(m[i], 0.0f) : m[i], l[i]);
        float* po = (DIRECT ? osm : ws.part_o) + ((size_t)rec * G + head) * D + 8 * g;
#pragma unroll
        for (int j = 0; j < JV; ++j) {
          float4* to = reinterpret_cast<float4*>(po + 64 * j);
          to[0] = make_float4(acc[j][0][i], acc[j][0][2 + i], acc[j][1][i], acc[j][1][2 + i]);
          to[1] = make_float4(acc[j][2][i], acc[j][2][2 + i], acc[j][3][i], acc[j][3][2 + i]);
        }
      }
    }
  };

  Chunk cur = look_up(lane), nxt = look_up(32 + lane);
  grid_dependency_wait();  // the pages: the write of this step's tokens may still run
  int row = __shfl_sync(0xffffffffu, cur.row, 0);
  load_k(row);
  load_v(row);
  int bh = DIRECT ? (int)blockIdx.x : __shfl_sync(0xffffffffu, cur.bh, 0);
  begin_pair(bh);
#pragma unroll 1
  for (int x = lo; x < hi; ++x) {
    const int i = (x - lo) & 31;
    const uint32_t mask = __shfl_sync(0xffffffffu, cur.mask, i);
    const int b1 = __shfl_sync(0xffffffffu, cur.bh, i);
    if (i == 31) {  // the next block of 32 chunks, looked up one block ago
      cur = nxt;
      nxt = look_up(x - lo + 33 + lane);
    }
    const int row1 = __shfl_sync(0xffffffffu, cur.row, (i + 1) & 31);  // of chunk x + 1
    if (b1 != bh) {
      end_pair(bh);
      bh = b1;
      begin_pair(bh);
    }
    float s[2][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) s[0][k] = s[1][k] = 0.0f;
    if (row >= 0) {
#pragma unroll
      for (int j = 0; j < JK; ++j) {
        if constexpr (Q32) {
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const uint4 q = *reinterpret_cast<const uint4*>(qw + (k * JK + j) * 512);
            mma_bf16(s[0], ka[j].x, kb[j].x, ka[j].y, kb[j].y, q.x, q.y);
            mma_bf16(s[1], ka[j].z, kb[j].z, ka[j].w, kb[j].w, q.z, q.w);
          }
        } else {
          mma_bf16(s[0], ka[j].x, kb[j].x, ka[j].y, kb[j].y, qf[j].x, qf[j].y);
          mma_bf16(s[1], ka[j].z, kb[j].z, ka[j].w, kb[j].w, qf[j].z, qf[j].w);
        }
      }
    }
    load_k(row1);
    if (row >= 0) {
      float y[4];  // (key g, head 2c), (g, 2c+1), (g+8, 2c), (g+8, 2c+1) in log2 units
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = (s[0][k] + s[1][k]) * sl;
      if (mask != 0xFFFFu) {
        if (!((mask >> g) & 1)) y[0] = y[1] = -CUDART_INF_F;
        if (!((mask >> (g + 8)) & 1)) y[2] = y[3] = -CUDART_INF_F;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (!((mask >> (2 * c + 8 * (k >> 1) + (k & 1))) & 1))
#pragma unroll
            for (int j = 0; j < JV; ++j) vr[k][j] = make_uint4(0, 0, 0, 0);
      }
      const float t0 = fmaxf(y[0], y[2]), t1 = fmaxf(y[1], y[3]);
      if (__any_sync(0xffffffffu, t0 > m[0] + D16_SLACK || t1 > m[1] + D16_SLACK)) {
        float t[2] = {t0, t1};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) t[k] = fmaxf(t[k], __shfl_xor_sync(0xffffffffu, t[k], o));
          const float mn = fmaxf(m[k], t[k]);
          const float f = m[k] == -CUDART_INF_F ? 0.0f : ex2(m[k] - mn);
          m[k] = mn;
          l[k] *= f;
#pragma unroll
          for (int j = 0; j < JV; ++j)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              acc[j][w][k] *= f;
              acc[j][w][2 + k] *= f;
            }
        }
      }
      const float m0 = m[0] == -CUDART_INF_F ? 0.0f : m[0], m1 = m[1] == -CUDART_INF_F ? 0.0f : m[1];
      const float p0 = ex2(y[0] - m0), p1 = ex2(y[1] - m1), p2 = ex2(y[2] - m0), p3 = ex2(y[3] - m1);
      l[0] += p0 + p2;
      l[1] += p1 + p3;
      uint32_t wlo[3], whi[3];  // the weights of keys 0-7 and 8-15, three terms
      split3(p0, p1, wlo);
      split3(p2, p3, whi);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        wlo[k] = transpose8x8(wlo[k]);
        whi[k] = transpose8x8(whi[k]);
      }
#pragma unroll
      for (int j = 0; j < JV; ++j) {
        const uint32_t v0[4] = {vr[0][j].x, vr[0][j].y, vr[0][j].z, vr[0][j].w};
        const uint32_t v1[4] = {vr[1][j].x, vr[1][j].y, vr[1][j].z, vr[1][j].w};
        const uint32_t v2[4] = {vr[2][j].x, vr[2][j].y, vr[2][j].z, vr[2][j].w};
        const uint32_t v3[4] = {vr[3][j].x, vr[3][j].y, vr[3][j].z, vr[3][j].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a0 = prmt(v0[w], v1[w], 0x5410), a1 = prmt(v0[w], v1[w], 0x7632);
          const uint32_t a2 = prmt(v2[w], v3[w], 0x5410), a3 = prmt(v2[w], v3[w], 0x7632);
          float o[4];  // of this chunk alone: see the header on the sums' rounding
          mma_bf16_fresh(o, a0, a1, a2, a3, wlo[0], whi[0]);
          mma_bf16(o, a0, a1, a2, a3, wlo[1], whi[1]);
          mma_bf16(o, a0, a1, a2, a3, wlo[2], whi[2]);
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[j][w][k] += o[k];
        }
      }
    }
    load_v(row1);
    row = row1;
  }
  end_pair(bh);
  err = __reduce_or_sync(0xffffffffu, err);
  if (err && lane == 0) flag_error(P.dev_error, err);
  if constexpr (DIRECT) {
    __syncthreads();
    for (int i = threadIdx.x; i < G * D / 4; i += NT) {
      const int head = i / (D / 4), d = 4 * (i % (D / 4));
      float M = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) M = fmaxf(M, mlsm[w * G + head].x);
      float sum = 0.0f;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float2 ml = mlsm[w * G + head];
        const float f = ml.x == -CUDART_INF_F ? 0.0f : ex2(ml.x - M);
        const float4 x = *reinterpret_cast<const float4*>(osm + (size_t)(w * G + head) * D + d);
        sum = fmaf(f, ml.y, sum);
        o.x = fmaf(f, x.x, o.x);
        o.y = fmaf(f, x.y, o.y);
        o.z = fmaf(f, x.z, o.z);
        o.w = fmaf(f, x.w, o.w);
      }
      const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;  // no visible key: zeros
      const size_t row = (size_t)(blockIdx.x / Hkv) * P.num_q_heads + (blockIdx.x % Hkv) * G + head;
      *reinterpret_cast<float4*>(P.out + row * D + d) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
  }
}

template <int N>
__device__ __forceinline__ void load_dims(const float* p, float (&v)[N]) {  // through L2: other SMs wrote them
  if constexpr (N == 4) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(p));
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else if constexpr (N == 2) {
    const float2 x = __ldcg(reinterpret_cast<const float2*>(p));
    v[0] = x.x; v[1] = x.y;
  } else {
    v[0] = __ldcg(p);
  }
}

// Joins the records of one (sequence, q head): W warps each take every W-th
// group of RPS records (running maximum, sum and output of their own, joined
// through shared memory); lane l holds EPL dims.  W = 1 when a pair is cut into
// few records (eight heads to a CTA), 8 or 32 when into many; with 32 each CTA
// takes 32 dims only, so that a call over one long sequence has CTAs enough to
// read its records at speed (one warp per head took 90 us over one sequence
// of 131071 keys, one CTA of 32 warps per head 11).
template <int D, int W>
__global__ void __launch_bounds__(W > 8 ? 32 * W : 256) decode16_merge_kernel(const AttnParams P, const DecodeWs ws) {
  constexpr int EPL = W > 8 ? 1 : D / 32;
  constexpr int CUTS = D / 32 / EPL;          // CTAs per head
  constexpr int HEADS = W > 8 ? 1 : 8 / W;    // heads per CTA
  constexpr int RPS = 8;                      // records per step
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % W;
  const long long wid = (long long)(blockIdx.x / CUTS) * HEADS + warp / W;
  const int d0 = (blockIdx.x % CUTS) * 32 * EPL + EPL * lane;  // the lane's first dim
  const int Hq = P.num_q_heads, G = P.group, Hkv = P.num_kv_heads;
  if (wid >= (long long)P.batch * Hq) return;  // (whole CTAs, for W > 1)
  const int b = (int)(wid / Hq), hq = (int)(wid % Hq), head = hq % G;
  const int bh = b * Hkv + hq / G, BH = P.batch * Hkv;
  grid_dependency_wait();  // every record is written
  const int T = __ldcg(ws.tile_start + BH);
  const int start = __ldcg(ws.tile_start + bh), end = __ldcg(ws.tile_start + bh + 1);
  float m = -CUDART_INF_F, l = 0.0f, o[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) o[e] = 0.0f;
  if (start < end && KVQ_IN_BOUNDS(start >= 0 && end <= T, P.dev_error)) {  // else no visible key: zeros
    const int nw = stream_workers(T, ws.nwall, ws.fixed_workers, D16_MIN_CHUNKS);
    const int w0 = worker_of(start, T, nw);
    int n = worker_of(end - 1, T, nw) - w0 + 1;
    if (!KVQ_IN_BOUNDS(w0 >= 0 && w0 + n - 1 + bh < ws.n_partials, P.dev_error)) n = 0;
    const size_t rec0 = (size_t)(w0 + bh) * G + head;
    for (int r0 = RPS * part; r0 < n; r0 += RPS * W) {
      float2 ml[RPS];
      float v[RPS][EPL];
#pragma unroll
      for (int u = 0; u < RPS; ++u) {  // the loads of a step in flight together
        const size_t rec = rec0 + (size_t)min(r0 + u, n - 1) * G;
        ml[u] = __ldcg(ws.part_ml + rec);
        load_dims<EPL>(ws.part_o + rec * D + d0, v[u]);
      }
      float mn = m;
#pragma unroll
      for (int u = 0; u < RPS; ++u)
        if (r0 + u < n && ml[u].y != 0.0f) mn = fmaxf(mn, ml[u].x);
      if (mn == -CUDART_INF_F) continue;  // nothing visible in these
      const float f = m == -CUDART_INF_F ? 0.0f : ex2(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) o[e] *= f;
#pragma unroll
      for (int u = 0; u < RPS; ++u) {
        if (r0 + u < n && ml[u].y != 0.0f) {
          const float x = ex2(ml[u].x - m);
          l = fmaf(x, ml[u].y, l);
#pragma unroll
          for (int e = 0; e < EPL; ++e) o[e] = fmaf(x, v[u][e], o[e]);
        }
      }
    }
  }
  if constexpr (W > 1) {
    __shared__ float sm_m[W], sm_l[W], sm_o[W][32 * EPL];
    if (lane == 0) {
      sm_m[part] = m;
      sm_l[part] = l;
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) sm_o[part][EPL * lane + e] = o[e];
    __syncthreads();
    if (part != 0) return;
    float M = m;
#pragma unroll
    for (int w = 1; w < W; ++w) M = fmaxf(M, sm_m[w]);
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float x = sm_m[w] == -CUDART_INF_F ? 0.0f : ex2(sm_m[w] - M);
      l = fmaf(x, sm_l[w], l);
#pragma unroll
      for (int e = 0; e < EPL; ++e) o[e] = fmaf(x, sm_o[w][EPL * lane + e], o[e]);
    }
  }
  float* out = P.out + (size_t)wid * D + d0;
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  if constexpr (EPL == 4) *reinterpret_cast<float4*>(out) = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
  else if constexpr (EPL == 2) *reinterpret_cast<float2*>(out) = make_float2(o[0] * inv, o[1] * inv);
  else *out = o[0] * inv;
}

size_t decode16_smem(int D, bool q32, bool direct, int group) {
  return (q32 ? (size_t)d16_warps(D) * 3 * (D / 32) * 512 : 0) + (direct ? (size_t)d16_warps(D) * group * (D * 4 + 8) : 0);
}

template <int D, bool Q32, bool DIRECT>
cudaError_t launch_decode16_t(const AttnParams& P, const DecodeWs& ws, int grid, cudaStream_t stream) {
  const int most = (int)decode16_smem(D, Q32, DIRECT, 8);
  if (most > 0) {
    // the opt-in shared-memory size is set once per device (not inside later
    // calls, which may be captured into a CUDA graph)
    static bool attr_set[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
      e = cudaFuncSetAttribute(decode16_kernel<D, Q32, DIRECT>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
  }
  return launch_dependent(decode16_kernel<D, Q32, DIRECT>, dim3(grid), dim3(d16_warps(D) * 32),
                          decode16_smem(D, Q32, DIRECT, P.group), stream, P, ws);
}

template <int D>
cudaError_t launch_decode16_d(const AttnParams& P, const DecodeWs& ws, int grid, cudaStream_t stream) {
  const bool f32 = P.dtype == DT_F32;
  const int pairs = P.batch * P.num_kv_heads;
  // One CTA per pair while that is short: a wave of CTAs costs about two chunks
  // of a warp's time and each chunk of its longest warp one, and the split form
  // with its second launch six (66 sequences of 2 keys, 264 pairs: 8.4 us).
  // What the host knows of the lengths is the table's width.
  const long long chunks = (long long)P.max_blocks * (P.block_size / D16_KEYS);  // of a pair, at most
  const long long waves = (pairs + grid - 1) / grid, per_warp = (chunks + d16_warps(D) - 1) / d16_warps(D);
  if (ws.fixed_workers == 0 && waves * (2 + per_warp) <= D16_DIRECT_COST)
    return f32 ? launch_decode16_t<D, true, true>(P, ws, pairs, stream)
               : launch_decode16_t<D, false, true>(P, ws, pairs, stream);
  cudaError_t e = f32 ? launch_decode16_t<D, true, false>(P, ws, grid, stream)
                      : launch_decode16_t<D, false, false>(P, ws, grid, stream);
  if (e != cudaSuccess) return e;
  const long long heads = (long long)P.batch * P.num_q_heads;
  // a pair is cut into nwall / pairs records on average when the GPU is full
  const long long cuts = chunks < ws.nwall / pairs ? chunks : ws.nwall / pairs;
  if (cuts >= 8 * D16_WIDE_MERGE)
    return launch_dependent(decode16_merge_kernel<D, 32>, dim3((unsigned)(heads * (D / 32))), dim3(1024), 0, stream, P, ws);
  if (cuts >= D16_WIDE_MERGE)
    return launch_dependent(decode16_merge_kernel<D, 8>, dim3((unsigned)heads), dim3(256), 0, stream, P, ws);
  return launch_dependent(decode16_merge_kernel<D, 1>, dim3((unsigned)((heads + 7) / 8)), dim3(256), 0, stream, P, ws);
}

}  // namespace

DecodeShape decode16_shape(int head_dim) { return {1, d16_warps(head_dim)}; }

cudaError_t launch_decode16(const AttnParams& P, const DecodeWs& ws, int grid, cudaStream_t stream) {
  return P.head_dim == 128 ? launch_decode16_d<128>(P, ws, grid, stream) : launch_decode16_d<64>(P, ws, grid, stream);
}

}  // namespace kvq
