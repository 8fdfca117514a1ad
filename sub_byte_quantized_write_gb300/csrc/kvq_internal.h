// kvq_internal.h -- kernel parameter blocks and launchers behind the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_common.cuh"
#include "kvq_rope.cuh"

namespace kvq {

struct WriteParams {
  uint8_t* k_pages;
  uint8_t* v_pages;
  int num_blocks, num_kv_heads, block_size, head_dim, mode;
  int stego;                  // INT4 rows whose pad is an fp32 scale carrying the zero point
  const int8_t* signs;
  float* ch_amax;
  int32_t* ch_ready;
  const int32_t* table;
  int headwise, max_blocks, batch;
  const int32_t* seq_lens;
  const int32_t* cu_new;
  const void* k;
  const void* v;
  int dtype, num_tokens;
  int32_t* dev_error;
  // gather: dense outputs [num_tokens][Hkv][D] of out_dtype (DT_F32 / DT_BF16)
  void* out_k;
  void* out_v;
  int out_dtype;
  // gather with the current chunk in full precision (NULL chunk_k: plain
  // gather): sequence b's last cu_chunk[b+1] - cu_chunk[b] positions come
  // from rows cu_chunk[b] .. of chunk_k / chunk_v [rows][Hkv][D] of chunk_dtype
  const void* chunk_k;
  const void* chunk_v;
  const int32_t* cu_chunk;
  int chunk_dtype;
  RopeArgs rope;  // K rows are turned before they are stored
};

// kvq_rope: rows of q and k turned to their positions (q or k NULL: none).
struct RopeRows {
  RopeArgs rope;
  const int32_t* seq_lens;
  const int32_t* cu;
  int batch, num_tokens, head_dim, dtype;
  const void* in[2];   // q, k: [num_tokens] tokens of heads[] rows, stride[] elements apart
  void* out[2];
  int heads[2];
  long long in_stride[2], out_stride[2];
  int tokens_per_cta;
  int32_t* dev_error;
};

// Shared by the decode and prefill kernels.
struct AttnParams {
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  int num_blocks, num_kv_heads, block_size, head_dim, mode;
  int stego;                  // INT4 rows whose pad is an fp32 scale carrying the zero point
  const int8_t* signs;        // NULL = RHT off
  const float* ch_amax;       // INT8: [2][Hkv][D]
  const int32_t* table;
  int headwise, max_blocks, batch;
  const int32_t* seq_lens;
  const int32_t* window;      // [Hkv] or NULL
  int sink;
  const void* q;
  int dtype, num_q_heads, group;
  float softmax_scale;
  float* out;
  int32_t* dev_error;
  // prefill
  const int32_t* cu_q;
  int total_q, max_q_per_seq;
  // dense prefill: sequence b's key j is row cu_kv[b] + j of k_pages / v_pages;
  // kv_map[0 | 1] view K / V as [rows][Hkv][D] bf16 in boxes of one 64-dim half
  // of 64 rows of one head, 128-byte swizzled.
  // decode (token-head modes): kv_map[0 | 1] view the K / V pool as 2-D tensors
  // of page chunks (decode_chunk_rows), one chunk per box row.
  const int32_t* cu_kv;
  int chunk_rows_total;   // decode: rows of the kv_map tensors (the kernel copies no row at or past it)
  // decode with the step's write (kvq_write_decode_attn): the preparation
  // kernel quantises and stores the new K / V rows [num_new][Hkv][D] of
  // new_dtype; sequence b's are rows cu_new[b] .. cu_new[b+1] - 1 (NULL new_k:
  // no write).  16-bit pages: the write is the launch in front of the decode.
  const void* new_k;
  const void* new_v;
  int new_dtype, num_new;
  const int32_t* cu_new;
  RopeArgs rope;          // the query and the new K rows are turned to their positions
  // cross attention: the queries of cu_q (at most max_q_per_seq of a sequence)
  // each see every key.  By the decode kernels: q_group > 0, and `group` counts
  // the slots of a pair, query i's head g in slot i * q_group + g.  By the
  // tensor-core kernels: cross = 1, and each query tile's keys are cut into `splits`
  // parts, with `part` (splits > 1) their records, as split_record lays them out.
  int q_group, cross, splits;
  float* part;
  int exact;  // decode kernels: not 0 for the calls with rope and cross attention (decode_tma_kernel's FORM)
  // cross attention over bf16 rows with bf16 queries: q_map views them as
  // [total_q][num_q_heads][D] in boxes of one 64-dim half of `group` heads of as
  // many queries as a row tile holds (q_tma 0: the kernel loads them itself)
  int q_tma;
  CUtensorMap kv_map[2];  // 128-byte aligned by its own declaration
  CUtensorMap q_map;
};

// Decode workspace (caller-owned scratch), carved by decode_ws_layout.
struct DecodeWs {
  int* tile_start;     // [B*Hkv + 1] first stream tile of each pair (written by the stream kernel's CTA 0)
  uint32_t* qfrag;     // [B*Hkv][32 lanes][NT * D/16 * 2] query B-operand images
  float4* qbg;         // [B*Hkv][4*NT] per-head logit constants (beta, gamma, key fold, 0)
  float2* part_ml;     // [n_partials][G] (running max in log2 units, sum of weights)
  float* part_o;       // [n_partials][G][D] unnormalised partial outputs
  int n_partials;      // stream workers + B*Hkv
  int nwall;           // stream warps launched
  int fixed_workers;   // > 0: use exactly this many workers
};

constexpr int PREFILL_ROWS = 128;  // (query, q head) rows of a prefill CTA

// Split-KV geometry shared by the host API and the kernels.
constexpr int DECODE_KEYS_PER_TILE = 32;
constexpr int DECODE_WARPS = 4;
constexpr int DECODE_MIN_TILES_PER_WARP = 8;

// How the stream kernel of one configuration is launched: CTAs per SM and
// warps per CTA.
struct DecodeShape {
  int ctas_per_sm, warps_per_cta;
};

struct DecodeLayout {
  size_t off_tile_start, off_qfrag, off_qbg, off_part_ml, off_part_o, total;
  int grid, nwall, n_partials;
};

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace layout for one decode call; sm_count * ctas_per_sm CTAs of
// warps_per_cta warps.
inline DecodeLayout decode_ws_layout(int batch, int num_kv_heads, int group, int head_dim, int sm_count,
                                     DecodeShape shape) {
  DecodeLayout L;
  const int BH = batch * num_kv_heads;
  const int NT = group <= 4 ? 1 : 2;
  L.grid = sm_count * shape.ctas_per_sm;
  L.nwall = L.grid * shape.warps_per_cta;
  L.n_partials = L.nwall + BH;
  size_t o = 0;
  L.off_tile_start = o; o = align256(o + (size_t)(BH + 1) * 4);
  L.off_qfrag = o;      o = align256(o + (size_t)BH * 32 * NT * (head_dim / 16) * 2 * 4);
  L.off_qbg = o;        o = align256(o + (size_t)BH * 4 * NT * 16);
  L.off_part_ml = o;    o = align256(o + (size_t)L.n_partials * group * 8);
  L.off_part_o = o;     o = align256(o + (size_t)L.n_partials * group * head_dim * 4);
  L.total = o;
  return L;
}

// Page copies in every layer's pools (kvq_pages.cu).
constexpr int PAGE_MAX_LAYERS = 128;
struct PageCopy {
  uint8_t* pool[2 * PAGE_MAX_LAYERS];  // K and V of each cache in turn
  int unit_bytes[PAGE_MAX_LAYERS];     // one page: all heads of a block, or one head's
  int num_layers, most_bytes;          // the largest unit_bytes
  int pieces, run;                     // copy steps per page, and per CTA and turn
  int units;                        // pages of a pool
  const int32_t* src;
  const int32_t* dst;
  int num_pairs;
  const int32_t* num_pairs_dev;     // the pairs' number on the device instead, where not NULL
  unsigned long long* turn;         // runs handed out beyond the first of each CTA, where not NULL
  int32_t* claim;                   // [units] scratch of kvq_copy_pages for long lists
  int32_t* dev_error;
};

// Fork and compact: tables, counters and scratch.  `spaces` sets of page
// numbers (1, or one per kv head), row b of space s at table row b * spaces + s.
struct PagePlan {
  const int32_t* table;
  const int32_t* seq_lens;
  int max_blocks, batch, headwise, spaces, num_blocks, num_kv_heads, block_size, bs_log2;
  const int32_t* parents;      // fork
  const int32_t* keep_tokens;
  const int32_t* new_tokens;
  const int32_t* pins;
  int new_batch;
  int32_t* new_table;
  int32_t* new_lens;
  int32_t* refs;               // [spaces][num_blocks]
  int32_t* page_map;           // compact: [spaces][num_blocks]
  int32_t* num_used;           // compact: [spaces]
  int32_t* dev_error;
  // scratch
  int32_t* owner;              // [spaces][num_blocks] lowest row ending in a page; compact: the pages that may move
  int32_t* list;               // [spaces][num_blocks] free pages; compact: the holes
  int32_t* task_count;
  int4* row_info;              // fork: [new_batch * spaces] kept tokens, with the new ones, partly filled last page or -1
  int32_t* row_ask;            // fork: [new_batch * spaces] 2 * pages asked for + whether the last page is copied
  int32_t* row_at;             // fork: [new_batch * spaces] first page of the row's share
  int32_t* loose;              // compact: [spaces] used pages that may move, and those of them that stay
  int32_t* below;
  int32_t* pair_src;
  int32_t* pair_dst;
  int32_t* num_pairs;          // compact: one
  unsigned long long* turn;    // compact: one, 0 for the copies
  long long most_pairs;        // entries of pair_src / pair_dst
};
constexpr int PAGE_TASK_UNITS = 1024;  // fewest pages a CTA ranks at a time: sizes task_count
constexpr int PAGE_SEG = 256;          // entries of a table row a warp takes at a time

constexpr int PAGE_COPY_PIECE = 4096;   // bytes of a page that a warp copies in one step, at most
constexpr int PAGE_COPY_LISTED = 2048;  // pairs up to which kvq_copy_pages needs no scratch

cudaError_t launch_copy_pages(const PageCopy& C, int sms, cudaStream_t stream);
cudaError_t launch_fork(const PagePlan& P, PageCopy C, int sms, cudaStream_t stream);
cudaError_t launch_compact(const PagePlan& P, PageCopy C, int sms, cudaStream_t stream);

// Records of split query tiles: per tile and part the PREFILL_ROWS_PER_CTA rows'
// unnormalised outputs [rows][D], then their (maximum in log2 units, sum) pairs.
__host__ __device__ constexpr long long split_record_floats(int head_dim) {
  return (long long)PREFILL_ROWS * (head_dim + 2);
}

DecodeShape decode_shape(int mode, int head_dim, int group);
// Key rows per page chunk that the decode's tensor copies move (16 or 8), or 0
// when the configuration reads its pages another way (INT8 per channel, bf16).
// The caller's tensor maps kv_map[0 | 1] view the K / V pool as 2-D tensors
// of such chunks: row (block * Hkv + head) * (block_size / rows) + chunk.
int decode_chunk_rows(int mode, int head_dim, int group);

cudaError_t launch_write(const WriteParams& P, cudaStream_t stream);
cudaError_t launch_gather(const WriteParams& P, cudaStream_t stream);
// rotary positions (kvq_rope.cu)
cudaError_t launch_rope(RopeRows R, int sms, cudaStream_t stream);
// The step's write over 16-bit pages with rope: turned K and plain V rows into
// the pages, and the turned queries [batch][num_q_heads][D] as fp32 to q_out
// (q NULL: the write alone).
cudaError_t launch_rope_write16(const WriteParams& P, const void* q, int q_dtype, int num_q_heads, float* q_out,
                                int sms, cudaStream_t stream);
cudaError_t launch_decode(const AttnParams& P, const DecodeWs& ws, int grid, cudaStream_t stream);
// the decode over 16-bit pages (kvq_decode16.cu), which launch_decode and
// decode_shape hand to
DecodeShape decode16_shape(int head_dim);
cudaError_t launch_decode16(const AttnParams& P, const DecodeWs& ws, int grid, cudaStream_t stream);
cudaError_t launch_prefill(const AttnParams& P, cudaStream_t stream);
// cross attention over bf16 rows (kvq_cross16.cu): dense (cu_kv, rows by
// kv_map) or in pages (table; kv_map views the pools as rows); chunk_rows_total
// counts the maps' rows.
cudaError_t launch_cross16(const AttnParams& P, cudaStream_t stream);
// cross attention over quantised pages (kvq_crossq.cu)
cudaError_t launch_crossq(const AttnParams& P, cudaStream_t stream);
// joins the records of split query tiles, qtiles of each (sequence, kv head)
cudaError_t launch_split_merge(const AttnParams& P, int qtiles, cudaStream_t stream);

// The prefill grid: x = query tiles of the longest chunk (PREFILL_ROWS_PER_CTA
// (query, q head) rows per CTA), y = kv heads, z = sequences.  Computed in 64
// bits so that no max_q_per_seq can wrap it; the host checks it against the
// launch limits before any launch.
constexpr int PREFILL_ROWS_PER_CTA = PREFILL_ROWS;
inline long long prefill_grid_x(int max_q_per_seq, int group) {
  const long long qb = PREFILL_ROWS_PER_CTA / group;
  return ((long long)max_q_per_seq + qb - 1) / qb;
}

// CTAs of the cross attention over bf16 rows per (sequence, kv head, part): two
// row tiles each, one with fp32 queries.
inline long long cross16_blocks(int max_q_per_seq, int group, bool f32) {
  const long long tiles = prefill_grid_x(max_q_per_seq, group);
  return f32 ? tiles : (tiles + 1) / 2;
}

}  // namespace kvq
