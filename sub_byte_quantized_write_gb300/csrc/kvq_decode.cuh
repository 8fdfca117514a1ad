// kvq_decode.cuh -- what the decode kernels share (the low-bit pages' in
// kvq_decode.cu, the 16-bit pages' in kvq_decode16.cu): the visible tiles of a
// (sequence, kv head) pair, the cut of the tiles into one slice per warp, the
// merge of a pair's partial records, and the programmatic launch.
#pragma once

#include <math_constants.h>

#include "kvq_internal.h"

namespace kvq {

// ---------------------------------------------------------------------------
// Visible tile list of one (sequence, kv head): tiles [0, ns) and [tw, n_total)
// when a sliding window leaves a gap after the sink tiles, else [0, n_total).

struct TileList {
  int L, Leff, W, ns, tw, n_total, n_virt;
  bool gap;
};

template <bool READ_ONLY = true>
__device__ __forceinline__ TileList tile_list(const AttnParams& P, int b, int h, bool flag_errors, int KT) {
  TileList t;
  int L = load_input<READ_ONLY>(P.seq_lens + b);
  if (L < 0) {
    if (flag_errors) flag_error(P.dev_error, DEVERR_SEQ_LEN);
    L = 0;
  }
  t.L = L;
  t.Leff = L;
  if (t.Leff > P.max_blocks * P.block_size) {
    if (flag_errors) flag_error(P.dev_error, DEVERR_TABLE_RANGE);
    t.Leff = P.max_blocks * P.block_size;
  }
  t.W = P.window ? load_input<READ_ONLY>(P.window + h) : 0;
  t.n_total = (t.Leff + KT - 1) / KT;
  t.ns = 0;
  t.tw = 0;
  t.gap = false;
  if (t.W > 0) {
    const int kw = (L - 1) - t.W + 1;  // first key inside the window of the query at L - 1
    if (kw > 0) {
      t.ns = (min(P.sink, t.Leff) + KT - 1) / KT;
      t.tw = kw / KT;
      t.gap = t.tw > t.ns;
    }
  }
  // (max: of a length past the table, the window may start behind the last tile)
  t.n_virt = t.gap ? t.ns + max(t.n_total - t.tw, 0) : t.n_total;
  return t;
}

__device__ __forceinline__ int tile_of(const TileList& t, int v) {
  return (t.gap && v >= t.ns) ? t.tw + (v - t.ns) : v;
}

// Number of stream warps actually used for T tiles: at least min_tiles each,
// or `fixed` of them, but no more than there are tiles (a warp without a tile
// writes no record, and the merge reads one from every warp of a pair's range).
__device__ __forceinline__ int stream_workers(int T, int nwall, int fixed, int min_tiles = DECODE_MIN_TILES_PER_WARP) {
  if (fixed > 0) return max(1, min(min(fixed, nwall), T));
  return max(1, min(nwall, T / min_tiles));
}
__device__ __forceinline__ int slice_lo(int w, int T, int nw) { return (int)((long long)w * T / nw); }
// The worker whose slice holds global tile x.
__device__ __forceinline__ int worker_of(int x, int T, int nw) {
  return min(nw - 1, (int)(((long long)(x + 1) * nw - 1) / T));
}

// ---------------------------------------------------------------------------
// merge helpers (used by the merge kernel)

// Merge records w0 + bh .. w0 + nrec - 1 + bh of q head i of pair bh
// (log-sum-exp weights), apply the output transform (inverse RHT with the
// signs tsign, or the INT8 V channel scales) and 1 / l, and store the D
// outputs at `out`; one warp, element d = lane + 32 e in lane `lane`.
// Records are read through L2 (they may come from other SMs of this grid).
template <int D>
__device__ __forceinline__ void merge_records(const AttnParams& P, const DecodeWs& ws, int bh, int i, int w0,
                                              int nrec, const float (&tsign)[D / 32], float* out, int lane) {
  constexpr int EPL = D / 32;
  const int G = P.group;
  float o[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) o[e] = 0.0f;
  // one round trip for the first 32 records' sums and the first four
  // records' outputs; lane j holds record w0 + j
  // every record index w0 + r + bh must lie in the workspace
  if (!KVQ_IN_BOUNDS(w0 >= 0 && nrec >= 1 && w0 + nrec - 1 + bh < ws.n_partials, P.dev_error)) nrec = 0;
  float2 ml0 = make_float2(-CUDART_INF_F, 0.0f);
  if (lane < nrec) ml0 = __ldcg(ws.part_ml + (size_t)(w0 + lane + bh) * G + i);
  constexpr int V0 = 8;  // records whose outputs load in the first round trip
  float v0[V0][EPL];
#pragma unroll
  for (int u = 0; u < V0; ++u) {
    const float* po = ws.part_o + ((size_t)(u < nrec ? w0 + u + bh : 0) * G + i) * D;
#pragma unroll
    for (int e = 0; e < EPL; ++e) v0[u][e] = u < nrec ? __ldcg(po + lane + 32 * e) : 0.0f;
  }
  float M = ml0.y > 0.0f ? ml0.x : -CUDART_INF_F;
  for (int j = 32 + lane; j < nrec; j += 32) {
    const float2 ml = __ldcg(ws.part_ml + (size_t)(w0 + j + bh) * G + i);
    if (ml.y > 0.0f) M = fmaxf(M, ml.x);
  }
  M = warp_max(M);
  if (M == -CUDART_INF_F) {
#pragma unroll
    for (int e = 0; e < EPL; ++e) out[lane + 32 * e] = 0.0f;
    return;
  }
  float l = 0.0f;
  for (int c0 = 0; c0 < nrec; c0 += 32) {
    float2 ml = ml0;
    if (c0 > 0) {
      ml = make_float2(-CUDART_INF_F, 0.0f);
      if (c0 + lane < nrec) ml = __ldcg(ws.part_ml + (size_t)(w0 + c0 + lane + bh) * G + i);
    }
    const float f = (c0 + lane < nrec && ml.y > 0.0f) ? ex2(ml.x - M) : 0.0f;
    l += f * ml.y;
    const int n = min(32, nrec - c0);
    int kfirst = 0;
    if (c0 == 0) {  // the first V0 records: outputs loaded with the sums above
#pragma unroll
      for (int u = 0; u < V0; ++u) {
        const float fk = __shfl_sync(0xffffffffu, f, u);
        const bool use = u < n && fk != 0.0f;
#pragma unroll
        for (int e = 0; e < EPL; ++e) o[e] = fmaf(use ? fk : 0.0f, use ? v0[u][e] : 0.0f, o[e]);
      }
      kfirst = V0;
    }
    // then four records per round, their loads issued together
    for (int k0 = kfirst; k0 < n; k0 += 4) {
      float fk[4];
      float v[4][EPL];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        fk[u] = __shfl_sync(0xffffffffu, f, (k0 + u) & 31);
        const bool use = k0 + u < n && fk[u] != 0.0f;
        const float* po = ws.part_o + ((size_t)(w0 + c0 + k0 + u + bh) * G + i) * D;
#pragma unroll
        for (int e = 0; e < EPL; ++e) v[u][e] = use ? __ldcg(po + lane + 32 * e) : 0.0f;
        if (!use) fk[u] = 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < EPL; ++e) o[e] = fmaf(fk[u], v[u][e], o[e]);
    }
  }
  l = warp_sum(l);
  // element d = lane + 32 e: lane bits are d bits 0-4, e bits are d bits 5-6
  if (P.mode != MODE_INT8 && P.signs) {
#pragma unroll
    for (int lm = 1; lm < 32; lm <<= 1) {
      const bool upper = (lane & lm) != 0;
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        const float x = __shfl_xor_sync(0xffffffffu, o[e], lm);
        o[e] = upper ? x - o[e] : o[e] + x;
      }
    }
#pragma unroll
    for (int hstep = 1; hstep < EPL; hstep <<= 1)
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        if (e & hstep) continue;
        const float a = o[e], c = o[e + hstep];
        o[e] = a + c;
        o[e + hstep] = a - c;
      }
    const float inv = 1.0f / ((float)D * l);
#pragma unroll
    for (int e = 0; e < EPL; ++e) out[lane + 32 * e] = tsign[e] * o[e] * inv;
  } else if (P.mode == MODE_INT8) {
#pragma unroll
    for (int e = 0; e < EPL; ++e) out[lane + 32 * e] = o[e] * tsign[e] / l;
  } else {
#pragma unroll
    for (int e = 0; e < EPL; ++e) out[lane + 32 * e] = o[e] / l;
  }
}

// Row of q and out of slot i (< P.group) of pair (b, h): the decode query's head
// i of the pair, or with P.q_group > 0 query i / q_group of the sequence; -1
// where it has no such query.  `flag`: report queries that are not served.
__device__ __forceinline__ long long slot_row(const AttnParams& P, int b, int h, int i, bool flag = false) {
  if (P.q_group == 0) return (long long)b * P.num_q_heads + h * P.group + i;
  const int c0 = load_input<false>(P.cu_q + b), n = load_input<false>(P.cu_q + b + 1) - c0;
  if (flag && (n > P.max_q_per_seq || (n > 0 && (c0 < 0 || c0 > P.total_q - n)))) flag_error(P.dev_error, DEVERR_SEQ_LEN);
  const int qi = i / P.q_group;
  if (qi >= n || c0 + qi < 0 || c0 + qi >= P.total_q) return -1;
  return (long long)(c0 + qi) * P.num_q_heads + h * P.q_group + i % P.q_group;
}

template <typename Kern, typename... Args>
cudaError_t launch_dependent(Kern kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace kvq
