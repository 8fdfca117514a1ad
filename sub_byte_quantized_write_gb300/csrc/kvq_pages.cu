// kvq_pages.cu -- pages as objects: copying them, giving new table rows the
// pages of parent rows (fork, which also frees and reserves), and moving the
// used ones to the lowest numbers (compact).
//
// A "space" is a set of page numbers 0 .. num_blocks - 1 with its own table
// rows: one for a uniform table (a block holds every kv head's page), one per
// kv head for a head-wise table.  Everything but the copying is whole-number
// work on tables and per-page counters, cheap in bytes and made of dependent
// phases (count the uses, rank the free pages, hand them out), so it is bound
// by latency: the phases run in one kernel, a cluster of 16 CTAs with the
// hardware's cluster barrier between phases, as long as a phase is short;
// past PLAN_FUSED_WORK elements each phase is a launch of its own over the
// whole GPU.  The page copies are a second launch over a list of (source,
// destination) pairs: bound by memory.  Where they can be no more than
// PLAN_COPIES bytes they are the cluster's last phase instead: 3 us less of the
// host's time per call against 1 us more on the GPU (four beams: 20.3 and 11.3
// against 23.5 and 10.7 us).  The border between the two forms of the plan: a
// fork over 93 thousand pages and entries takes 18.9 us in a cluster and 20.5
// in launches, over 233 thousand 29 and 20.
//
// What bounds the plan is its chain of loads: per phase one or two trips to L2
// and the barrier's flush (1.2 thousand cycles of 2 to 5 thousand, by clock
// stamps).  Sixteen CTAs against eight, with one page per thread, and counters
// loaded before they are looked at: 19 us for 64 searches of 4 beams against 28.
//
// Nothing depends on the order in which atomics land: counters only add, the
// owner of a shared last page is a minimum, and page numbers are handed out
// by prefix sums (the k-th request in row order gets the k-th lowest free
// page).

#include <climits>

#include "kvq_decode.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_CLUSTER = 8;
constexpr long long PLAN_FUSED_WORK = 1 << 17;  // pages and table entries
constexpr long long PLAN_COPIES = 2 << 20;      // bytes of page copies that the plan's CTAs do themselves
// A task, the pages that a CTA ranks at a time, has ITEMS consecutive pages per
// thread: one (coalesced; every CTA of the cluster busy) up to PLAN_SMALL
// tasks, four beyond.
constexpr int PLAN_SMALL = 128;
static_assert(PAGE_TASK_UNITS == PLAN_THREADS, "task_count has one entry per task of one page per thread");

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive prefix sum over the CTA's PLAN_THREADS threads, and the total.
// Every thread calls it.  `sm` holds two sets of 33 ints, used in turn, so
// that a call needs no barrier before it writes.
struct BlockScan {
  int (*sm)[33];
  int turn = 0;
  __device__ __forceinline__ int operator()(int v, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int* a = sm[turn];
    turn ^= 1;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) a[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      const int t = a[lane];
      int s = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      a[lane] = s - t;
      if (lane == 31) a[32] = s;
    }
    __syncthreads();
    total = a[32];
    return a[warp] + incl - v;
  }
};

// Sum of a[0 .. n - 1], by every warp for itself.
__device__ __forceinline__ int warp_total(const int* a, int n) {
  int v = 0;
  for (int i = threadIdx.x & 31; i < n; i += 32) v += __ldcg(a + i);
  return __reduce_add_sync(0xffffffffu, v);
}

// Consecutive counters from `first` on; those at or past n read as `past`.
template <int ITEMS>
__device__ __forceinline__ void load_items(const int32_t* a, int first, int n, int past, int (&x)[ITEMS]) {
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) x[i] = first + i < n ? __ldcg(a + first + i) : past;
}

// Page `id` of space `s` as a number of the pools: blocks for a uniform
// table, (block, head) pages for a head-wise one.
__device__ __forceinline__ int pool_unit(const PagePlan& P, int s, int id) {
  return P.spaces == 1 && !P.headwise ? id : id * P.num_kv_heads + s;
}

// Copies.  One warp copies one piece (up to COPY_PIECE bytes) of page s of one
// pool into page d at a time: eight 16-byte loads per lane in flight, then the
// stores.  Step `item` of a pair: pool item / pieces, piece item % pieces.
constexpr int COPY_PIECE = PAGE_COPY_PIECE;

template <int LOADS>  // in flight per lane
__device__ __forceinline__ void copy_piece(const PageCopy& P, int s, int d, int item) {
  const int lane = threadIdx.x & 31;
  const int lk = item / P.pieces, piece = item - lk * P.pieces, bytes = P.unit_bytes[lk >> 1];
  const int size = ((bytes + P.pieces - 1) / P.pieces + 15) & ~15, lo = piece * size, n = min(size, bytes - lo);
  const uint8_t* from = P.pool[lk] + (size_t)s * bytes + lo;
  uint8_t* to = P.pool[lk] + (size_t)d * bytes + lo;
#pragma unroll 1
  for (int at = 16 * lane; at < n; at += 512 * LOADS) {
    uint4 x[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k)
      if (at + 512 * k < n) x[k] = *reinterpret_cast<const uint4*>(from + at + 512 * k);
#pragma unroll
    for (int k = 0; k < LOADS; ++k)
      if (at + 512 * k < n) *reinterpret_cast<uint4*>(to + at + 512 * k) = x[k];
  }
}

// The pairs of a plan, by the plan's own CTAs.
__device__ void copy_planned(const PagePlan& P, const PageCopy& C) {
  const int pairs = P.num_pairs ? __ldcg(P.num_pairs) : P.new_batch * P.spaces;
  const int per_pair = 2 * C.num_layers * C.pieces, items = pairs * per_pair;  // (few: see PLAN_COPIES)
  for (int w = blockIdx.x * (PLAN_THREADS / 32) + (threadIdx.x >> 5); w < items; w += gridDim.x * (PLAN_THREADS / 32)) {
    const int i = w / per_pair, s = __ldcg(P.pair_src + i), d = __ldcg(P.pair_dst + i);
    if (s >= 0 && d >= 0) copy_piece<4>(C, s, d, w - i * per_pair);
  }
}

// ---------------------------------------------------------------------------
// fork

struct ForkRow {
  int parent;       // -1: a row that starts empty
  int kept, total;  // tokens of the parent that stay, and with the new ones
};

__device__ __forceinline__ ForkRow fork_row(const PagePlan& P, int b, int& err) {
  ForkRow r;
  r.parent = __ldg(P.parents + b);
  r.kept = r.total = 0;
  if (r.parent >= P.batch) {
    err |= DEVERR_ROW_RANGE;
    r.parent = -1;
    return r;
  }
  if (r.parent < 0) r.parent = -1;
  const long long cap = min((long long)P.max_blocks * P.block_size, (long long)INT_MAX);
  long long L = r.parent >= 0 ? __ldg(P.seq_lens + r.parent) : 0;
  if (L < 0) err |= DEVERR_SEQ_LEN;
  if (L > cap) err |= DEVERR_TABLE_RANGE;
  L = max(0LL, min(L, cap));
  if (P.keep_tokens) {
    const long long k = __ldg(P.keep_tokens + b);
    if (k < 0) err |= DEVERR_SEQ_LEN;
    L = min(L, max(0LL, k));
  }
  long long n = P.new_tokens ? __ldg(P.new_tokens + b) : 0;
  if (n < 0) err |= DEVERR_SEQ_LEN;
  n = L + max(0LL, n);
  if (n > cap) err |= DEVERR_TABLE_RANGE;
  r.kept = (int)L;
  r.total = (int)min(n, cap);
  return r;
}

__device__ __forceinline__ int pages_of(const PagePlan& P, int tokens) {
  return (tokens >> P.bs_log2) + ((tokens & (P.block_size - 1)) != 0);
}

// Phase 0: the counters.
__device__ void fork_init(const PagePlan& P) {
  const long long n = (long long)P.spaces * P.num_blocks;
  for (long long u = (long long)blockIdx.x * PLAN_THREADS + threadIdx.x; u < n; u += (long long)gridDim.x * PLAN_THREADS) {
    P.refs[u] = P.pins ? max(0, __ldg(P.pins + u)) : 0;
    P.owner[u] = INT_MAX;
  }
}

// Phase 1: the kept entries of every new row; their uses counted.  A partly
// filled last page is not counted but claimed, by the lowest row that ends in
// it.  row_info: what the later phases need of a row.
__device__ void fork_mark(const PagePlan& P) {
  constexpr int SEG = PAGE_SEG;  // entries of a row per warp and step
  const int lane = threadIdx.x & 31;
  const int segs = (P.max_blocks + SEG - 1) / SEG;
  const int tasks = P.new_batch * P.spaces * segs, step = gridDim.x * (PLAN_THREADS / 32);
  int err = 0;
  for (int t = blockIdx.x * (PLAN_THREADS / 32) + (threadIdx.x >> 5); t < tasks; t += step) {
    const int r = t / segs, e0 = (t - r * segs) * SEG;
    const int b = r / P.spaces, s = r - b * P.spaces;
    const ForkRow row = fork_row(P, b, err);
    if (s == 0 && e0 == 0 && lane == 0) P.new_lens[b] = row.total;
    const int have = pages_of(P, row.kept), tail = row.kept & (P.block_size - 1) ? have - 1 : -1;
    const int32_t* from = P.table + ((long long)row.parent * P.spaces + s) * P.max_blocks;
    int32_t* to = P.new_table + (long long)r * P.max_blocks;
    int v[SEG / 32];
#pragma unroll
    for (int k = 0; k < SEG / 32; ++k) {
      const int e = e0 + lane + 32 * k;
      v[k] = e < have ? __ldg(from + e) : -1;
    }
    if (e0 == 0 && lane == 0 && tail < 0) P.row_info[r] = make_int4(row.kept, row.total, -1, 0);
#pragma unroll
    for (int k = 0; k < SEG / 32; ++k) {
      const int e = e0 + lane + 32 * k;
      if (v[k] >= P.num_blocks) err |= DEVERR_BLOCK_RANGE;
      if (v[k] < 0 || v[k] >= P.num_blocks) v[k] = -1;
      if (e < P.max_blocks) to[e] = v[k];
      if (e == tail) P.row_info[r] = make_int4(row.kept, row.total, v[k], 0);
      if (v[k] >= 0) {
        const long long u = (long long)s * P.num_blocks + v[k];
        if (e == tail) atomicMin(P.owner + u, b);
        else atomicAdd(P.refs + u, 1);
      }
    }
  }
  err = __reduce_or_sync(0xffffffffu, err);
  if (err && lane == 0) flag_error(P.dev_error, err);
}

// Bit i: page first + i of space s is free.
template <int ITEMS>
__device__ __forceinline__ int fork_free(const PagePlan& P, int s, int first) {
  int refs[ITEMS], owner[ITEMS], f = 0;
  load_items(P.refs + (long long)s * P.num_blocks, first, P.num_blocks, 1, refs);
  load_items(P.owner + (long long)s * P.num_blocks, first, P.num_blocks, 0, owner);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) f |= (refs[i] == 0 && owner[i] == INT_MAX) << i;
  return f;
}

// Phase 2: free pages per task, and the pages each row asks for: a private
// copy of its last page unless it is the lowest row that ends in it and
// nobody else uses it, and pages for its new tokens.
template <int ITEMS>
__device__ void fork_count(const PagePlan& P, BlockScan& scan) {
  const int rows = P.new_batch * P.spaces;
  for (int r = blockIdx.x * PLAN_THREADS + threadIdx.x; r < rows; r += gridDim.x * PLAN_THREADS) {
    const int b = r / P.spaces, s = r - b * P.spaces;
    const int4 row = __ldcg(P.row_info + r);  // kept, total, last page
    int split = 0;
    if (row.z >= 0) {
      const long long u = (long long)s * P.num_blocks + row.z;
      const int refs = __ldcg(P.refs + u), owner = __ldcg(P.owner + u);
      split = refs > 0 || owner != b;
    }
    P.row_ask[r] = 2 * (pages_of(P, row.y) - pages_of(P, row.x) + split) + split;
  }
  constexpr int UNITS = ITEMS * PLAN_THREADS;
  const int per_space = (P.num_blocks + UNITS - 1) / UNITS;
  for (int t = blockIdx.x; t < P.spaces * per_space; t += gridDim.x) {
    const int s = t / per_space, first = (t - s * per_space) * UNITS + ITEMS * threadIdx.x;
    int total;
    scan(__popc(fork_free<ITEMS>(P, s, first)), total);
    if (threadIdx.x == 0) P.task_count[t] = total;
  }
}

// Phase 3: the free pages of each space in ascending order, and where each
// row's share of them begins (rows in order).
template <int ITEMS>
__device__ void fork_rank(const PagePlan& P, BlockScan& scan) {
  constexpr int UNITS = ITEMS * PLAN_THREADS;
  const int per_space = (P.num_blocks + UNITS - 1) / UNITS;
  for (int t = blockIdx.x; t < P.spaces * (per_space + 1); t += gridDim.x) {
    if (t < P.spaces * per_space) {
      const int s = t / per_space, k = t - s * per_space, first = k * UNITS + ITEMS * threadIdx.x;
      const int f = fork_free<ITEMS>(P, s, first);
      const int before = warp_total(P.task_count + s * per_space, k);
      int total;
      int at = before + scan(__popc(f), total);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (((f >> i) & 1) && KVQ_IN_BOUNDS(at < P.num_blocks, P.dev_error))
          P.list[(long long)s * P.num_blocks + at++] = first + i;
    } else {
      const int s = t - P.spaces * per_space;
      int before = 0;
      for (int b0 = 0; b0 < P.new_batch; b0 += PLAN_THREADS) {
        const int b = b0 + threadIdx.x;
        const int n = b < P.new_batch ? __ldcg(P.row_ask + (long long)b * P.spaces + s) >> 1 : 0;
        int total;
        const int at = before + scan(n, total);
        if (b < P.new_batch) P.row_at[(long long)b * P.spaces + s] = at;
        before += total;
      }
    }
  }
}

// Phase 4: the pages handed out, a warp per row; the pairs to copy.
template <int ITEMS>
__device__ void fork_assign(const PagePlan& P) {
  const int lane = threadIdx.x & 31;
  constexpr int UNITS = ITEMS * PLAN_THREADS;
  const int per_space = (P.num_blocks + UNITS - 1) / UNITS;
  const int rows = P.new_batch * P.spaces;
  int err = 0;
  for (int r = blockIdx.x * (PLAN_THREADS / 32) + (threadIdx.x >> 5); r < rows; r += gridDim.x * (PLAN_THREADS / 32)) {
    const int s = r % P.spaces;
    const int4 row = __ldcg(P.row_info + r);
    const int ask = __ldcg(P.row_ask + r), split = ask & 1, n = ask >> 1, at = __ldcg(P.row_at + r);
    const int n_free = warp_total(P.task_count + s * per_space, per_space);
    int32_t* to = P.new_table + (long long)r * P.max_blocks;
    int32_t* refs = P.refs + (long long)s * P.num_blocks;
    const int32_t* list = P.list + (long long)s * P.num_blocks;
    const int have = pages_of(P, row.x);
    int src = -1, dst = -1;
    for (int j = lane; j < n; j += 32) {
      const int id = at + j < n_free ? __ldcg(list + at + j) : -1;
      if (id < 0) err |= DEVERR_NO_PAGES;
      else refs[id] = 1;
      to[have + j - split] = id;  // the copy of the last page first, then the new ones
      if (split && j == 0 && id >= 0) {
        src = pool_unit(P, s, row.z);
        dst = pool_unit(P, s, id);
      }
    }
    if (lane == 0) {
      if (!split && row.z >= 0) refs[row.z] = 1;  // its only use (nothing pins it either, or it were split)
      P.pair_src[r] = src;
      P.pair_dst[r] = dst;
    }
  }
  err = __reduce_or_sync(0xffffffffu, err);
  if (err && lane == 0) flag_error(P.dev_error, err);
}

constexpr int FORK_PHASES = 5;

template <int ITEMS>
__global__ void __launch_bounds__(PLAN_THREADS, 1)
    fork_plan_kernel(const PagePlan P, const PageCopy C, int first, int last, bool copies_follow) {
  __shared__ int sm[2][33];
  BlockScan scan{sm};
  // The copies may launch; they wait for this grid to finish.
  if (copies_follow) allow_dependent_launch();
  for (int phase = first; phase <= last; ++phase) {
    if (phase == 0) fork_init(P);
    else if (phase == 1) fork_mark(P);
    else if (phase == 2) fork_count<ITEMS>(P, scan);
    else if (phase == 3) fork_rank<ITEMS>(P, scan);
    else if (phase == 4) fork_assign<ITEMS>(P);
    else copy_planned(P, C);
    if (phase < last) {
      __syncthreads();
      cluster_barrier();
    }
  }
}

// ---------------------------------------------------------------------------
// compact: with n pages of a space in use, a used page numbered n or above
// (a mover, unless pinned) moves into an unused page below n (a hole), the
// k-th mover into the k-th hole, both in ascending order.

__device__ void compact_init(const PagePlan& P) {
  const long long n = (long long)P.spaces * P.num_blocks;
  for (long long u = (long long)blockIdx.x * PLAN_THREADS + threadIdx.x; u < n; u += (long long)gridDim.x * PLAN_THREADS)
    P.refs[u] = P.pins ? max(0, __ldg(P.pins + u)) : 0;
}

// The entries of the table that count, those below a sequence's last token:
// f(index in the table, space, entry or -1) for every entry.
template <typename F>
__device__ __forceinline__ void compact_entries(const PagePlan& P, bool report, F f) {
  constexpr int SEG = PAGE_SEG;
  const int lane = threadIdx.x & 31;
  const int segs = (P.max_blocks + SEG - 1) / SEG;
  const int tasks = P.batch * P.spaces * segs, step = gridDim.x * (PLAN_THREADS / 32);
  const long long cap = (long long)P.max_blocks * P.block_size;
  int err = 0;
  for (int t = blockIdx.x * (PLAN_THREADS / 32) + (threadIdx.x >> 5); t < tasks; t += step) {
    const int r = t / segs, e0 = (t - r * segs) * SEG;
    const int b = r / P.spaces, s = r - b * P.spaces;
    const long long L = __ldg(P.seq_lens + b);
    if (L < 0) err |= DEVERR_SEQ_LEN;
    if (L > cap) err |= DEVERR_TABLE_RANGE;
    const int have = pages_of(P, (int)max(0LL, min(L, cap)));
    const long long i0 = (long long)r * P.max_blocks;
    int v[SEG / 32];
#pragma unroll
    for (int k = 0; k < SEG / 32; ++k) {
      const int e = e0 + lane + 32 * k;
      v[k] = e < P.max_blocks ? __ldcg(P.table + i0 + e) : -1;
      if (e >= have) v[k] = -1;
    }
#pragma unroll
    for (int k = 0; k < SEG / 32; ++k) {
      const int e = e0 + lane + 32 * k;
      if (v[k] >= P.num_blocks) err |= DEVERR_BLOCK_RANGE;
      if (e < P.max_blocks) f(i0 + e, s, v[k] < 0 || v[k] >= P.num_blocks ? -1 : v[k]);
    }
  }
  err = __reduce_or_sync(0xffffffffu, err);
  if (report && err && lane == 0) flag_error(P.dev_error, err);
}

__device__ void compact_mark(const PagePlan& P) {
  compact_entries(P, true, [&](long long, int s, int v) {
    if (v >= 0) atomicAdd(P.refs + (long long)s * P.num_blocks + v, 1);
  });
}

// Pages first .. first + ITEMS - 1 of space s: bit i, page first + i is used; bit 4 + i, and not pinned.
template <int ITEMS>
__device__ __forceinline__ int compact_used(const PagePlan& P, int s, int first) {
  int refs[ITEMS], pins[ITEMS] = {}, f = 0;
  load_items(P.refs + (long long)s * P.num_blocks, first, P.num_blocks, 0, refs);
  if (P.pins) load_items(P.pins + (long long)s * P.num_blocks, first, P.num_blocks, 0, pins);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    f |= (refs[i] > 0) << i;
    f |= (refs[i] > 0 && pins[i] <= 0) << (4 + i);
  }
  return f;
}

// Phase 2: used pages per task, and the used ones that may move.  (Both in
// one scan: a task has at most 4096 of each.)
template <int ITEMS>
__device__ void compact_count(const PagePlan& P, BlockScan& scan) {
  constexpr int UNITS = ITEMS * PLAN_THREADS;
  const int per_space = (P.num_blocks + UNITS - 1) / UNITS;
  const int tasks = P.spaces * per_space;
  for (int t = blockIdx.x; t < tasks; t += gridDim.x) {
    const int s = t / per_space, first = (t - s * per_space) * UNITS + ITEMS * threadIdx.x;
    const int f = compact_used<ITEMS>(P, s, first);
    int total;
    scan(__popc(f & 15) + (__popc(f >> 4) << 16), total);
    if (threadIdx.x == 0) {
      P.task_count[t] = total & 0xFFFF;
      P.task_count[tasks + t] = total >> 16;
    }
  }
}

// Phase 3: every page's rank: the holes listed in order, and the used pages
// that may move (those numbered n_used or above are the movers; `below` is how
// many of the list come before them), the map of all that stay.
template <int ITEMS>
__device__ void compact_rank(const PagePlan& P, BlockScan& scan) {
  constexpr int UNITS = ITEMS * PLAN_THREADS;
  const int per_space = (P.num_blocks + UNITS - 1) / UNITS;
  const int tasks = P.spaces * per_space;
  for (int t = blockIdx.x; t < tasks; t += gridDim.x) {
    const int s = t / per_space, k = t - s * per_space, first = k * UNITS + ITEMS * threadIdx.x;
    const long long u0 = (long long)s * P.num_blocks;
    const int f = compact_used<ITEMS>(P, s, first);
    const int n_used = warp_total(P.task_count + s * per_space, per_space);
    int ru = warp_total(P.task_count + s * per_space, k);
    int rl = warp_total(P.task_count + tasks + s * per_space, k);
    int total;
    const int in = scan(__popc(f & 15) + (__popc(f >> 4) << 16), total);
    if (k == per_space - 1 && threadIdx.x == 0) {
      P.num_used[s] = n_used;
      P.loose[s] = rl + (total >> 16);
      if (n_used == P.num_blocks) P.below[s] = rl + (total >> 16);
    }
    ru += in & 0xFFFF;
    rl += in >> 16;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int id = first + i;
      if (id >= P.num_blocks) break;
      const bool used = (f >> i) & 1, may = (f >> (4 + i)) & 1;
      if (id == n_used) P.below[s] = rl;
      if (!used && id < n_used && KVQ_IN_BOUNDS(ru <= id, P.dev_error))
        P.list[u0 + id - ru] = id;  // hole: as many holes before it as unused pages
      if (may && KVQ_IN_BOUNDS(rl < P.num_blocks, P.dev_error)) P.owner[u0 + rl] = id;
      if (!may || id < n_used) P.page_map[u0 + id] = used ? id : -1;
      ru += used;
      rl += may;
    }
  }
}

// Phase 4: the movers' new numbers, their counts moved, the pairs to copy
// (the spaces' one after another).
__device__ void compact_pair(const PagePlan& P) {
  int before = 0;
  for (int s = 0; s < P.spaces; ++s) {
    const int below = __ldcg(P.below + s), n = __ldcg(P.loose + s) - below;
    const long long u0 = (long long)s * P.num_blocks;
    for (int k = blockIdx.x * PLAN_THREADS + threadIdx.x; k < n; k += gridDim.x * PLAN_THREADS) {
      const int src = __ldcg(P.owner + u0 + below + k), dst = __ldcg(P.list + u0 + k);
      if (!KVQ_IN_BOUNDS(dst >= 0 && dst < src && src < P.num_blocks && before + k < P.most_pairs, P.dev_error)) continue;
      P.page_map[u0 + src] = dst;
      P.refs[u0 + dst] = __ldcg(P.refs + u0 + src);
      P.refs[u0 + src] = 0;
      P.pair_src[before + k] = pool_unit(P, s, src);
      P.pair_dst[before + k] = pool_unit(P, s, dst);
    }
    before += n;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *P.num_pairs = before;
    *P.turn = 0;
  }
}

__device__ void compact_remap(const PagePlan& P) {
  compact_entries(P, false, [&](long long i, int s, int v) {
    P.new_table[i] = v >= 0 ? __ldcg(P.page_map + (long long)s * P.num_blocks + v) : -1;
  });
}

constexpr int COMPACT_PHASES = 6;

template <int ITEMS>
__global__ void __launch_bounds__(PLAN_THREADS, 1)
    compact_plan_kernel(const PagePlan P, const PageCopy C, int first, int last, bool copies_follow) {
  __shared__ int sm[2][33];
  BlockScan scan{sm};
  // The copies may launch; they wait for this grid to finish.
  if (copies_follow) allow_dependent_launch();
  for (int phase = first; phase <= last; ++phase) {
    if (phase == 0) compact_init(P);
    else if (phase == 1) compact_mark(P);
    else if (phase == 2) compact_count<ITEMS>(P, scan);
    else if (phase == 3) compact_rank<ITEMS>(P, scan);
    else if (phase == 4) compact_pair(P);
    else if (phase == 5) compact_remap(P);
    else copy_planned(P, C);
    if (phase < last) {
      __syncthreads();
      cluster_barrier();
    }
  }
}

// ---------------------------------------------------------------------------
// copies

// claim[page] = -1 for a page that some pair reads, else the lowest pair that
// writes it.  Only the entries the pairs name are set, so the array need not
// be cleared.
__global__ void __launch_bounds__(PLAN_THREADS, 1) copy_claim_kernel(const PageCopy P) {
  allow_dependent_launch();  // the copies may launch; they wait for this grid to finish
  const int n = P.num_pairs, step = gridDim.x * PLAN_THREADS, i0 = blockIdx.x * PLAN_THREADS + threadIdx.x;
  for (int i = i0; i < n; i += step) {
    const int s = __ldg(P.src + i), d = __ldg(P.dst + i);
    if (s < 0 || d < 0 || s >= P.units || d >= P.units) continue;
    P.claim[s] = INT_MAX;
    P.claim[d] = INT_MAX;
  }
  __syncthreads();
  cluster_barrier();
  for (int i = i0; i < n; i += step) {
    const int s = __ldg(P.src + i), d = __ldg(P.dst + i);
    if (s < 0 || d < 0 || s >= P.units || d >= P.units) continue;
    atomicMin(P.claim + s, -1);
    if (s != d) atomicMin(P.claim + d, i);
  }
}

// A CTA takes a run of consecutive pieces of one pair.  Bound by memory: 1200
// pages of 32 layers, 1.34 GB read and written, 197 us alone, the rate of a
// plain copy; of COPY_RUN 16, 32 and 64, and of one CTA per run (or runs taken
// in turn where the device alone knows their number) against fixed strides,
// these measured fastest (226 us for the compaction of 96 sequences against 234).
// How a pair is known to be free of conflicts: by construction (fork, compact),
// by the claims of the kernel before, or, for short lists, by the CTA itself,
// which compares the pair with the whole list: that saves a launch, 12 of 221 us
// for 1200 pages of 32 layers and 2 us of the host's time for a few pages.
// (Measured and not kept for pages of 2 KB or less, one head's of a low-bit
// cache, which leave most of a warp's loads empty: a step over several pools,
// with the page's bytes laid end to end or pool by pool: 91 and 97 us instead
// of 78 for 126,000 pages of 1152 bytes.)
// Where a pair has fewer steps than a run (few layers, small pages) a run spans
// several pairs, each warp looking up its own (ONE_PAIR false): 660 thousand
// pages of 320 bytes in one layer, 630 us instead of 2030.  Not so for short
// lists: checked by warps, 468 pages of one layer took 7.5 us instead of 4.8.
constexpr int COPY_RUN = 16;  // copy steps per CTA and turn; twice that over several pairs
enum { COPY_SAFE, COPY_CLAIMED, COPY_CHECKS_LIST };

template <int CHECK, bool ONE_PAIR>
__global__ void __launch_bounds__(256) copy_pages_kernel(const PageCopy P) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (CHECK != COPY_CHECKS_LIST) grid_dependency_wait();  // the pairs come from the kernel before
  const long long pairs = P.num_pairs_dev ? __ldcg(P.num_pairs_dev) : P.num_pairs;
  const int per_pair = 2 * P.num_layers * P.pieces;
  // runs: of each pair, or of all pairs' steps end to end
  const int runs_pp = (per_pair + P.run - 1) / P.run;
  const long long steps = pairs * per_pair, runs = ONE_PAIR ? pairs * runs_pp : (steps + P.run - 1) / P.run;
  __shared__ unsigned long long turn[2];
  int phase = 0;
  auto next = [&](long long w) -> long long {  // the CTA's next run
    if (!P.turn) return w + gridDim.x;
    if (threadIdx.x == 0) turn[phase] = gridDim.x + atomicAdd(P.turn, 1ull);
    __syncthreads();
    phase ^= 1;
    return (long long)turn[phase ^ 1];
  };
  long long i = -1;  // the pair looked up last, by the CTA (ONE_PAIR) or the warp: page s into page d
  int s = -1, d = -1;
  auto look_up = [&](long long pair, bool reports) -> bool {  // whether to copy it
    i = pair;
    s = __ldcg(P.src + i);
    d = __ldcg(P.dst + i);
    if (s < 0 || d < 0 || s == d) return false;
    if (s >= P.units || d >= P.units) {
      if (reports) flag_error(P.dev_error, DEVERR_BLOCK_RANGE);
      return false;
    }
    bool conflict = false;  // read by another pair, or written by a lower one
    if (CHECK == COPY_CLAIMED) conflict = __ldcg(P.claim + d) != (int)i;
    if constexpr (CHECK == COPY_CHECKS_LIST) {
      static_assert(ONE_PAIR, "the CTA compares its one pair with the list");
      int hit = 0;
      for (int j = threadIdx.x; j < P.num_pairs; j += 256) {
        const int a = __ldg(P.src + j), b = __ldg(P.dst + j);
        hit |= a >= 0 && b >= 0 && a < P.units && b < P.units && (a == d || (b == d && a != b && j < i));
      }
      conflict = __syncthreads_or(hit);
    }
    if (conflict && reports) flag_error(P.dev_error, DEVERR_PAGE_CONFLICT);
    return !conflict;
  };
  for (long long w = blockIdx.x; w < runs; w = next(w)) {
    if constexpr (ONE_PAIR) {
      const int first = (int)(w % runs_pp) * P.run, last = min(first + P.run, per_pair);
      if (!look_up(w / runs_pp, first == 0 && threadIdx.x == 0)) continue;
      for (int item = first + warp; item < last; item += 8) copy_piece<COPY_PIECE / 512>(P, s, d, item);
    } else {
      const long long last = min((w + 1) * P.run, steps);
      bool go = false;
      for (long long item = w * P.run + warp; item < last; item += 8) {
        const long long pair = item / per_pair;
        if (pair != i) go = look_up(pair, lane == 0);
        if (go) copy_piece<COPY_PIECE / 512>(P, s, d, (int)(item - pair * per_pair));
      }
      i = -1;
    }
  }
}

// ---------------------------------------------------------------------------
// launch

// A cluster of sixteen CTAs where the device can hold one (more than eight is
// for a kernel to opt in to), else of eight.  Asked once per kernel and device,
// not inside later calls, which may be captured into a graph.
template <typename Kern, typename... Args>
cudaError_t launch_cluster(Kern kernel, int (&sizes)[64], cudaStream_t stream, Args... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(PLAN_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int size = dev < 64 ? sizes[dev] : PLAN_CLUSTER;
  if (size == 0) {
    attr[0].val.clusterDim.x = 2 * PLAN_CLUSTER;
    cfg.gridDim = dim3(2 * PLAN_CLUSTER);
    int n = 0;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) (void)cudaGetLastError();  // (a refusal of the larger size is no error of this call)
    size = e == cudaSuccess && n > 0 ? 2 * PLAN_CLUSTER : PLAN_CLUSTER;
    sizes[dev] = size;
  }
  attr[0].val.clusterDim.x = size;
  cfg.gridDim = dim3(size);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool small_plan(const PagePlan& P) {
  return (long long)P.spaces * ((P.num_blocks + PLAN_THREADS - 1) / PLAN_THREADS) <= PLAN_SMALL;
}

template <int CHECK>
cudaError_t launch_copies(PageCopy C, long long most_pairs, int sms, cudaStream_t stream) {
  const long long per_pair = 2LL * C.num_layers * C.pieces;
  const long long resident = (long long)sms * 4;
  // long runs when there are steps enough to fill the GPU with them, else one step per warp
  C.run = most_pairs * per_pair < resident * COPY_RUN ? 8 : per_pair < COPY_RUN ? 2 * COPY_RUN : COPY_RUN;
  const bool one_pair = CHECK == COPY_CHECKS_LIST || per_pair >= C.run;
  const long long ctas =
      one_pair ? most_pairs * ((per_pair + C.run - 1) / C.run) : (most_pairs * per_pair + C.run - 1) / C.run;
  if (ctas == 0) return cudaSuccess;
  // one CTA per run where the host knows their number, else as many as fit,
  // which take their runs in turn
  const dim3 grid((unsigned)(ctas < resident || (!C.turn && ctas <= INT_MAX) ? ctas : resident));
  if constexpr (CHECK == COPY_CHECKS_LIST) {  // nothing before it to overlap with
    copy_pages_kernel<CHECK, true><<<grid, 256, 0, stream>>>(C);
    return cudaGetLastError();
  } else {
    return one_pair ? launch_dependent(copy_pages_kernel<CHECK, true>, grid, dim3(256), 0, stream, C)
                    : launch_dependent(copy_pages_kernel<CHECK, false>, grid, dim3(256), 0, stream, C);
  }
}

// The phases of a plan and the copies: in one launch, in two, or, for large
// plans, in one per phase and the copies'.
template <typename Kern>
cudaError_t launch_plan(Kern kernel, int (&sizes)[64], const PagePlan& P, const PageCopy& C, int phases, int sms,
                        cudaStream_t stream) {
  const long long rows = (long long)(P.new_batch > P.batch ? P.new_batch : P.batch) * P.spaces;
  const long long work = (long long)P.spaces * P.num_blocks + rows * P.max_blocks;
  if (work <= PLAN_FUSED_WORK) {
    const bool copies = P.most_pairs * 2 * C.num_layers * C.most_bytes <= PLAN_COPIES;
    const cudaError_t e = launch_cluster(kernel, sizes, stream, P, C, 0, copies ? phases : phases - 1, !copies);
    if (e != cudaSuccess || copies) return e;
  } else {
    for (int i = 0; i < phases; ++i) {
      kernel<<<sms, PLAN_THREADS, 0, stream>>>(P, C, i, i, i == phases - 1 && P.most_pairs > 0);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
  }
  return launch_copies<COPY_SAFE>(C, P.most_pairs, sms, stream);
}

}  // namespace

cudaError_t launch_copy_pages(const PageCopy& C, int sms, cudaStream_t stream) {
  if (C.num_pairs <= PAGE_COPY_LISTED) return launch_copies<COPY_CHECKS_LIST>(C, C.num_pairs, sms, stream);
  static int sizes[64] = {0};
  const cudaError_t e = launch_cluster(copy_claim_kernel, sizes, stream, C);
  if (e != cudaSuccess) return e;
  return launch_copies<COPY_CLAIMED>(C, C.num_pairs, sms, stream);
}

cudaError_t launch_fork(const PagePlan& P, PageCopy C, int sms, cudaStream_t stream) {
  static int sizes[2][64] = {{0}, {0}};
  C.src = P.pair_src;
  C.dst = P.pair_dst;
  C.num_pairs = P.new_batch * P.spaces;
  return small_plan(P) ? launch_plan(fork_plan_kernel<1>, sizes[0], P, C, FORK_PHASES, sms, stream)
                       : launch_plan(fork_plan_kernel<4>, sizes[1], P, C, FORK_PHASES, sms, stream);
}

cudaError_t launch_compact(const PagePlan& P, PageCopy C, int sms, cudaStream_t stream) {
  static int sizes[2][64] = {{0}, {0}};
  C.src = P.pair_src;
  C.dst = P.pair_dst;
  C.num_pairs_dev = P.num_pairs;
  C.turn = P.turn;
  return small_plan(P) ? launch_plan(compact_plan_kernel<1>, sizes[0], P, C, COMPACT_PHASES, sms, stream)
                       : launch_plan(compact_plan_kernel<4>, sizes[1], P, C, COMPACT_PHASES, sms, stream);
}

}  // namespace kvq
