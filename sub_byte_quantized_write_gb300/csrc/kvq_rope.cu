// kvq_rope.cu -- rotary positions: rows of q and k turned to their positions
// (kvq_rope), and a step's write over 16-bit pages with its queries.
//
// (a, b) -> A (a c - b s, b c + a s) for each pair of a row, the pairs either
// half the turned dims apart or neighbours; see kvq_rope.cuh for the angles.
// Three multiplies and adds per element against two bytes in and two out:
// bound by memory, or for a few tokens by the launch and the chain token ->
// sequence -> position.
//
// One CTA takes a few tokens.  Its first threads find their positions, all of
// them the cosines and sines, each pair of each token once and for all heads
// (a table in shared memory: worked out per head they would cost more than
// the rows' bytes do), and then each thread turns pieces of 16 elements, with
// the loads of its first pieces issued before any of that.  Measured: 8192 tokens
// of 32 + 8 heads of 128 dims in bf16 34.9 us, 4.8 TB/s (71% of a copy's rate; what
// is missing are the CTAs' starts); one token 2.5 us on the GPU.
//
// The rotary positions of a layer's projections come before the cache write
// of the pages' sources: vLLM PR #40835 review summary, 实现拆解 item 2 (the
// write kernel takes the K and V rows as the layer has turned them).

#include <algorithm>

#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int ROPE_TOKENS = 8;  // of a CTA, at most
constexpr int ROPE_PIECE = 16;  // elements per step of a thread

// Position of token t by the write's map; false for a token outside every
// sequence, or of a sequence with more new tokens than its length.
__device__ __forceinline__ bool token_position(const int32_t* cu, const int32_t* seq_lens, int batch, int t, int& pos,
                                               int& seq, int32_t* dev_error) {
  int lo = 0, hi = batch - 1;  // the last sequence whose first token is <= t
  // a decode step's one token per sequence is where it is first looked for
  if (t < batch && __ldg(cu + t) <= t && t < __ldg(cu + t + 1)) lo = hi = t;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  const int c0 = __ldg(cu + lo), c1 = __ldg(cu + lo + 1);
  if (t < c0 || t >= c1) return false;
  const int L = __ldg(seq_lens + lo);
  if (L < 0 || c1 - c0 > L) {
    flag_error(dev_error, DEVERR_SEQ_LEN);
    return false;
  }
  pos = L - (c1 - c0) + (t - c0);
  seq = lo;
  return true;
}

// Where the two blocks of eight elements of piece `pc` of a row start: the
// elements and their partners, or (interleaved pairs, dims that do not turn)
// two neighbouring blocks.
__device__ __forceinline__ void piece_dims(const RopeArgs& R, int pc, int& a, int& b) {
  const bool split = !R.inter && ROPE_PIECE * pc < R.rot;
  a = split ? 8 * pc : ROPE_PIECE * pc;
  b = split ? a + R.rot / 2 : a + 8;
}

// Turns the 16 elements of piece `pc` (x[0]: from dim a on, x[1]: from b on)
// by the token's table of cosines and sines; pieces past the turned dims stay.
__device__ __forceinline__ void turn_piece(const RopeArgs& R, const float2* table, int pc, float (&x)[2][8]) {
  if (ROPE_PIECE * pc >= R.rot) return;
  const float4* w4 = reinterpret_cast<const float4*>(table + 8 * pc);  // pairs 8 pc .. + 7, either way
  if (R.inter) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 w = w4[k];
      float(&v)[8] = x[k >> 1];
      const int e = 4 * (k & 1);
      const float p = v[e], q = v[e + 1], r = v[e + 2], t = v[e + 3];
      v[e] = fmaf(p, w.x, q * -w.y);
      v[e + 1] = fmaf(q, w.x, p * w.y);
      v[e + 2] = fmaf(r, w.z, t * -w.w);
      v[e + 3] = fmaf(t, w.z, r * w.w);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 w = w4[k];
      const float p = x[0][2 * k], q = x[1][2 * k], r = x[0][2 * k + 1], t = x[1][2 * k + 1];
      x[0][2 * k] = fmaf(p, w.x, q * -w.y);
      x[1][2 * k] = fmaf(q, w.x, p * w.y);
      x[0][2 * k + 1] = fmaf(r, w.z, t * -w.w);
      x[1][2 * k + 1] = fmaf(t, w.z, r * w.w);
    }
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool F32>
__device__ __forceinline__ void store8(void* out, long long at, const float (&x)[8]) {
  if constexpr (F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = pack8(x);
  }
}

// The tables of a CTA's tokens, for those whose `valid` is set.
template <int D>
__device__ __forceinline__ void fill_tables(const RopeArgs& R, int tokens, const int* pos, float2 (*table)[D / 2]) {
  const int pairs = R.rot / 2;
  for (int i = threadIdx.x; i < tokens * (D / 2); i += blockDim.x) {
    const int k = i / (D / 2), p = i % (D / 2);
    if (p >= pairs) continue;
    const float2 w = rope_cos_sin(rope_turns(__ldg(R.inv_freq + p)), pos[k]);
    table[k][p] = make_float2(w.x * R.scale, w.y * R.scale);
  }
}

// Eight elements as they lie in memory: 16 bytes of bf16, 32 of fp32.
template <bool F32>
struct Raw8 {
  uint4 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw8<F32> load_raw8(const void* in, long long at) {
  Raw8<F32> r;
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i)  // (plain loads: the output may be the input)
    r.w[i] = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(in) + at * (F32 ? 4 : 2))[i];
  return r;
}
template <bool F32>
__device__ __forceinline__ void store_raw8(void* out, long long at, const Raw8<F32>& r) {
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + at * (F32 ? 4 : 2))[i] = r.w[i];
}
template <bool F32>
__device__ __forceinline__ void unpack8(const Raw8<F32>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) {
    const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (F32) {
        x[4 * i + k] = __uint_as_float(w[k]);
      } else {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    }
  }
}

template <int D, bool F32>
__global__ void __launch_bounds__(256, 6) rope_kernel(const RopeRows R) {
  constexpr int PPR = D / ROPE_PIECE;  // pieces per row
  constexpr int U = 1;                 // pieces in flight per thread
  __shared__ __align__(16) float2 table[ROPE_TOKENS][D / 2];
  __shared__ int pos[ROPE_TOKENS];
  __shared__ int valid[ROPE_TOKENS];
  const int t0 = blockIdx.x * R.tokens_per_cta, tokens = min(R.tokens_per_cta, R.num_tokens - t0);
  const int heads = R.heads[0] + R.heads[1];
  const int items = tokens * heads * PPR;
  // item i: piece i % PPR of head i / PPR % heads (q's, then k's) of token i / PPR / heads
  struct Item {
    int tok, head, a, b;
  };
  auto item = [&](int i) -> Item {
    Item it;
    const int r = i / PPR;
    it.tok = r / heads;
    it.head = r % heads;
    piece_dims(R.rope, i % PPR, it.a, it.b);
    return it;
  };
  Raw8<F32> x[U][2];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 256;
      if (i >= items) break;
      const Item it = item(i);
      const int k = it.head >= R.heads[0];
      const long long at = (long long)(t0 + it.tok) * R.in_stride[k] + (it.head - (k ? R.heads[0] : 0)) * D;
      x[u][0] = load_raw8<F32>(R.in[k], at + it.a);
      x[u][1] = load_raw8<F32>(R.in[k], at + it.b);
    }
  };
  fetch(threadIdx.x);
  if (threadIdx.x < tokens) {
    int p = 0, seq = 0;
    const int t = t0 + threadIdx.x;
    bool ok = true;
    if (R.rope.positions) p = __ldg(R.rope.positions + t);
    else ok = token_position(R.cu, R.seq_lens, R.batch, t, p, seq, R.dev_error);
    pos[threadIdx.x] = p;
    valid[threadIdx.x] = ok;
  }
  __syncthreads();
  fill_tables<D>(R.rope, tokens, pos, table);
  __syncthreads();
  for (int i0 = threadIdx.x;; i0 += U * 256) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 256;
      if (i >= items) break;
      const Item it = item(i);
      if (!valid[it.tok]) continue;
      const int k = it.head >= R.heads[0];
      const long long at = (long long)(t0 + it.tok) * R.out_stride[k] + (it.head - (k ? R.heads[0] : 0)) * D;
      if (ROPE_PIECE * (i % PPR) < R.rope.rot) {
        float f[2][8];
        unpack8<F32>(x[u][0], f[0]);
        unpack8<F32>(x[u][1], f[1]);
        turn_piece(R.rope, table[it.tok], i % PPR, f);
        store8<F32>(R.out[k], at + it.a, f[0]);
        store8<F32>(R.out[k], at + it.b, f[1]);
      } else {
        store_raw8<F32>(R.out[k], at + it.a, x[u][0]);
        store_raw8<F32>(R.out[k], at + it.b, x[u][1]);
      }
    }
    if (i0 + U * 256 >= items) break;
    fetch(i0 + U * 256);
  }
}

// A step's write over 16-bit pages: blockIdx.y 0 takes the new tokens' K rows
// (turned) and V rows into the pages, 1 the queries (one per sequence, at the
// position of its last token) into q_out as fp32, from where the decode reads
// them.
template <int D>
__global__ void __launch_bounds__(256) rope_write16_kernel(const WriteParams P, const void* q, int q_dtype,
                                                           int num_q_heads, float* q_out, int tokens_per_cta) {
  constexpr int PPR = D / ROPE_PIECE;
  __shared__ __align__(16) float2 table[ROPE_TOKENS][D / 2];
  __shared__ int pos[ROPE_TOKENS], page_pos[ROPE_TOKENS], seqs[ROPE_TOKENS], valid[ROPE_TOKENS];
  allow_dependent_launch();  // a decode call after this write may launch now; it waits for this grid
  const bool queries = blockIdx.y == 1;
  const int total = queries ? P.batch : P.num_tokens;
  const int t0 = blockIdx.x * tokens_per_cta, tokens = min(tokens_per_cta, total - t0);
  if (tokens <= 0) return;
  if (threadIdx.x < tokens) {
    int p = 0, angle = 0, seq = t0 + threadIdx.x;
    bool ok = true;
    if (queries) {
      p = angle = __ldg(P.seq_lens + seq) - 1;
      if (P.rope.positions && P.num_tokens > 0) {
        const int c0 = __ldg(P.cu_new + seq), c1 = __ldg(P.cu_new + seq + 1);
        if (c1 > c0 && c1 >= 1 && c1 <= P.num_tokens) angle = __ldg(P.rope.positions + c1 - 1);
      }
    } else {
      const int t = t0 + threadIdx.x;
      ok = token_position(P.cu_new, P.seq_lens, P.batch, t, p, seq, P.dev_error);
      angle = P.rope.positions ? __ldg(P.rope.positions + t) : p;
    }
    pos[threadIdx.x] = angle;
    page_pos[threadIdx.x] = p;
    seqs[threadIdx.x] = seq;
    valid[threadIdx.x] = ok;
  }
  __syncthreads();
  fill_tables<D>(P.rope, tokens, pos, table);
  __syncthreads();
  const int heads = queries ? num_q_heads : P.num_kv_heads;
  const int items = tokens * heads * PPR;
  for (int i = threadIdx.x; i < items; i += 256) {
    const int pc = i % PPR, r = i / PPR, k = r / heads, h = r % heads;
    int a, b;
    piece_dims(P.rope, pc, a, b);
    float x[2][8];
    if (queries) {
      const long long row = ((long long)(t0 + k) * heads + h) * D;
      load_row_elems<8>(q, q_dtype, row + a, x[0]);
      load_row_elems<8>(q, q_dtype, row + b, x[1]);
      turn_piece(P.rope, table[k], pc, x);
      store8<true>(q_out, row + a, x[0]);
      store8<true>(q_out, row + b, x[1]);
      continue;
    }
    if (!valid[k]) continue;
    const long long row = ((long long)(t0 + k) * heads + h) * D;
    float v[2][8];
    load_row_elems<8>(P.k, P.dtype, row + a, x[0]);  // issued before the table entry is known
    load_row_elems<8>(P.k, P.dtype, row + b, x[1]);
    load_row_elems<8>(P.v, P.dtype, row + a, v[0]);
    load_row_elems<8>(P.v, P.dtype, row + b, v[1]);
    const int p = page_pos[k], lb = p / P.block_size;
    if (lb >= P.max_blocks) {
      if (pc == 0) flag_error(P.dev_error, DEVERR_TABLE_RANGE);
      continue;
    }
    const int blk = __ldg(P.table + (size_t)(P.headwise ? seqs[k] * P.num_kv_heads + h : seqs[k]) * P.max_blocks + lb);
    if (blk < 0) continue;  // evicted slot: nothing is written
    if (blk >= P.num_blocks) {
      if (pc == 0) flag_error(P.dev_error, DEVERR_BLOCK_RANGE);
      continue;
    }
    const size_t slot = ((size_t)blk * P.num_kv_heads + h) * P.block_size + p % P.block_size;
    if (!KVQ_IN_BOUNDS(slot < (size_t)P.num_blocks * P.num_kv_heads * P.block_size, P.dev_error)) continue;
    turn_piece(P.rope, table[k], pc, x);
    const long long at = (long long)slot * D;
    store8<false>(P.k_pages, at + a, x[0]);
    store8<false>(P.k_pages, at + b, x[1]);
    store8<false>(P.v_pages, at + a, v[0]);
    store8<false>(P.v_pages, at + b, v[1]);
  }
}

// Tokens per CTA: enough CTAs for every SM while the tokens are few, then as
// many tokens as keep the tables cheap.
int rope_tokens(long long tokens, int sms) {
  int n = 1;
  while (n < ROPE_TOKENS && tokens / (2 * n) >= 8LL * sms) n *= 2;
  return n;
}

template <int D>
cudaError_t launch_rope_d(const RopeRows& R, cudaStream_t stream) {
  const unsigned blocks = (unsigned)((R.num_tokens + (long long)R.tokens_per_cta - 1) / R.tokens_per_cta);
  if (R.dtype == DT_F32) rope_kernel<D, true><<<blocks, 256, 0, stream>>>(R);
  else rope_kernel<D, false><<<blocks, 256, 0, stream>>>(R);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(RopeRows R, int sms, cudaStream_t stream) {
  R.tokens_per_cta = rope_tokens(R.num_tokens, sms);
  return R.head_dim == 128 ? launch_rope_d<128>(R, stream) : launch_rope_d<64>(R, stream);
}

cudaError_t launch_rope_write16(const WriteParams& P, const void* q, int q_dtype, int num_q_heads, float* q_out,
                                int sms, cudaStream_t stream) {
  const long long most = std::max<long long>(P.num_tokens, q ? P.batch : 0);
  const int n = rope_tokens(most, sms);
  const dim3 grid((unsigned)((most + n - 1) / n), q ? 2 : 1);
  if (P.head_dim == 128) rope_write16_kernel<128><<<grid, 256, 0, stream>>>(P, q, q_dtype, num_q_heads, q_out, n);
  else rope_write16_kernel<64><<<grid, 256, 0, stream>>>(P, q, q_dtype, num_q_heads, q_out, n);
  return cudaGetLastError();
}

}  // namespace kvq
