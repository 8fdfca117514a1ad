// kvq_pages.cu -- pages as objects: copying them, giving new table rows the
// pages of parent rows (fork, which also frees and reserves), and moving the
// used ones to the lowest numbers (compact).
//
// A "space" is a set of page numbers 0 .. num_blocks - 1 with its own table
// rows: one for a uniform table (a block holds every kv head's page), one per
// kv head for a head-wise table.  Everything but the copying is whole-number
// work on tables and per-page counters, cheap in bytes and made of dependent
// phases (count the uses, rank the free pages, hand them out), so it is bound
// by latency: the phases run in one kernel, a cluster of eight CTAs with the
// hardware's cluster barrier between phases, as long as a phase is short;
// past PLAN_FUSED_WORK elements each phase is a launch of its own over the
// whole GPU.  The page copies are a second launch over a list of (source,
// destination) pairs: bound by memory.
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
constexpr long long PLAN_FUSED_WORK = 1 << 20;
constexpr int UNITS_PER_TASK = PAGE_TASK_UNITS;  // four per thread
static_assert(UNITS_PER_TASK == 4 * PLAN_THREADS, "four pages per thread");

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive prefix sum over the CTA's PLAN_THREADS threads, and the total.
// Every thread calls it; `sm` holds 33 ints.
__device__ __forceinline__ int block_scan(int v, int* sm, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // sm is free again
  if (lane == 31) sm[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int t = sm[lane];
    int s = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sm[lane] = s - t;
    if (lane == 31) sm[32] = s;
  }
  __syncthreads();
  total = sm[32];
  return sm[warp] + incl - v;
}

__device__ __forceinline__ int block_sum(const int* a, int n, int* sm) {  // of a[0 .. n - 1]
  int v = 0, total;
  for (int i = threadIdx.x; i < n; i += PLAN_THREADS) v += __ldcg(a + i);
  block_scan(v, sm, total);
  return total;
}

// Page `id` of space `s` as a number of the pools: blocks for a uniform
// table, (block, head) pages for a head-wise one.
__device__ __forceinline__ int pool_unit(const PagePlan& P, int s, int id) {
  return P.spaces == 1 && !P.headwise ? id : id * P.num_kv_heads + s;
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
  return tokens / P.block_size + (tokens % P.block_size != 0);
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
// filled last page is not counted but claimed, by the lowest row that ends in it.
__device__ void fork_mark(const PagePlan& P) {
  constexpr int SEG = 128;  // entries of a row per warp and step
  const int lane = threadIdx.x & 31;
  const int segs = (P.max_blocks + SEG - 1) / SEG;
  const long long tasks = (long long)P.new_batch * P.spaces * segs;
  int err = 0;
  for (long long t = (long long)blockIdx.x * (PLAN_THREADS / 32) + (threadIdx.x >> 5); t < tasks;
       t += (long long)gridDim.x * (PLAN_THREADS / 32)) {
    const long long r = t / segs;
    const int b = (int)(r / P.spaces), s = (int)(r % P.spaces), e0 = (int)(t % segs) * SEG;
    const ForkRow row = fork_row(P, b, err);
    if (s == 0 && e0 == 0 && lane == 0) P.new_lens[b] = row.total;
    const int have = pages_of(P, row.kept), tail = row.kept % P.block_size ? row.kept / P.block_size : -1;
    const int32_t* from = P.table + ((long long)row.parent * P.spaces + s) * P.max_blocks;
    int v[SEG / 32];
#pragma unroll
    for (int k = 0; k < SEG / 32; ++k) {
      const int e = e0 + lane + 32 * k;
      v[k] = e < have ? __ldg(from + e) : -1;
    }
#pragma unroll
    for (int k = 0; k < SEG / 32; ++k) {
      const int e = e0 + lane + 32 * k;
      if (v[k] >= P.num_blocks) err |= DEVERR_BLOCK_RANGE;
      if (v[k] < 0 || v[k] >= P.num_blocks) v[k] = -1;
      if (e < P.max_blocks) P.new_table[r * P.max_blocks + e] = v[k];
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

__device__ __forceinline__ bool fork_is_free(const PagePlan& P, long long u) {
  return __ldcg(P.refs + u) == 0 && __ldcg(P.owner + u) == INT_MAX;
}

// Phase 2: free pages per task, and the pages each row asks for: a private
// copy of its last page unless it is the lowest row that ends in it and
// nobody else uses it, and pages for its new tokens.
__device__ void fork_count(const PagePlan& P, int* sm) {
  const int per_space = (P.num_blocks + UNITS_PER_TASK - 1) / UNITS_PER_TASK;
  for (int t = blockIdx.x; t < P.spaces * per_space; t += gridDim.x) {
    const int s = t / per_space, first = (t % per_space) * UNITS_PER_TASK + 4 * threadIdx.x;
    int n = 0, total;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (first + i < P.num_blocks && fork_is_free(P, (long long)s * P.num_blocks + first + i)) ++n;
    block_scan(n, sm, total);
    if (threadIdx.x == 0) P.task_count[t] = total;
  }
  int err = 0;
  const long long rows = (long long)P.new_batch * P.spaces;
  for (long long r = (long long)blockIdx.x * PLAN_THREADS + threadIdx.x; r < rows; r += (long long)gridDim.x * PLAN_THREADS) {
    const int b = (int)(r / P.spaces), s = (int)(r % P.spaces);
    const ForkRow row = fork_row(P, b, err);
    int split = 0;
    if (row.kept % P.block_size) {
      const int v = __ldcg(P.new_table + r * P.max_blocks + row.kept / P.block_size);
      if (v >= 0) {
        const long long u = (long long)s * P.num_blocks + v;
        split = __ldcg(P.refs + u) > 0 || __ldcg(P.owner + u) != b;
      }
    }
    P.row_ask[r] = 2 * (pages_of(P, row.total) - pages_of(P, row.kept) + split) + split;
  }
}

// Phase 3: the free pages of each space in ascending order, and where each
// row's share of them begins (rows in order).
__device__ void fork_rank(const PagePlan& P, int* sm) {
  const int per_space = (P.num_blocks + UNITS_PER_TASK - 1) / UNITS_PER_TASK;
  for (int t = blockIdx.x; t < P.spaces * (per_space + 1); t += gridDim.x) {
    if (t < P.spaces * per_space) {
      const int s = t / per_space, k = t % per_space, first = k * UNITS_PER_TASK + 4 * threadIdx.x;
      const int before = block_sum(P.task_count + s * per_space, k, sm);
      bool free[4];
      int n = 0, total;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        free[i] = first + i < P.num_blocks && fork_is_free(P, (long long)s * P.num_blocks + first + i);
        n += free[i];
      }
      int at = before + block_scan(n, sm, total);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (free[i] && KVQ_IN_BOUNDS(at < P.num_blocks, P.dev_error)) P.list[(long long)s * P.num_blocks + at++] = first + i;
    } else {
      const int s = t - P.spaces * per_space;
      int before = 0;
      for (int b0 = 0; b0 < P.new_batch; b0 += PLAN_THREADS) {
        const int b = b0 + threadIdx.x;
        const long long r = (long long)b * P.spaces + s;
        const int n = b < P.new_batch ? __ldcg(P.row_ask + r) >> 1 : 0;
        int total;
        const int at = before + block_scan(n, sm, total);
        if (b < P.new_batch) P.row_at[r] = at;
        before += total;
      }
    }
  }
}

// Phase 4: the pages handed out, a warp per row; the pairs to copy.
__device__ void fork_assign(const PagePlan& P, int* sm) {
  const int lane = threadIdx.x & 31;
  const int per_space = (P.num_blocks + UNITS_PER_TASK - 1) / UNITS_PER_TASK;
  const long long rows = (long long)P.new_batch * P.spaces;
  int err = 0;
  // the number of free pages of each space, in turn (a warp's rows may be of any space)
  for (int s = 0; s < P.spaces; ++s) {
    const int n_free = block_sum(P.task_count + s * per_space, per_space, sm);
    for (long long w = (long long)blockIdx.x * (PLAN_THREADS / 32) + (threadIdx.x >> 5); w * P.spaces + s < rows;
         w += (long long)gridDim.x * (PLAN_THREADS / 32)) {
      const int b = (int)w;
      const long long r = w * P.spaces + s;
      const ForkRow row = fork_row(P, b, err);
      const int ask = __ldcg(P.row_ask + r), split = ask & 1, n = ask >> 1, at = __ldcg(P.row_at + r);
      int32_t* to = P.new_table + r * P.max_blocks;
      const int have = pages_of(P, row.kept);
      const int32_t* list = P.list + (long long)s * P.num_blocks;
      if (lane == 0) {
        int src = -1, dst = -1;
        if (row.kept % P.block_size) {
          const int v = __ldcg(to + have - 1);
          if (split) {
            const int id = at < n_free ? __ldcg(list + at) : -1;
            if (id < 0) err |= DEVERR_NO_PAGES;
            to[have - 1] = id;
            if (id >= 0) {
              P.refs[(long long)s * P.num_blocks + id] = 1;
              src = pool_unit(P, s, v);
              dst = pool_unit(P, s, id);
            }
          } else if (v >= 0) {
            P.refs[(long long)s * P.num_blocks + v] = 1;  // its only use (nothing pins it either, or it were split)
          }
        }
        P.pair_src[r] = src;
        P.pair_dst[r] = dst;
      }
      for (int j = split + lane; j < n; j += 32) {
        const int id = at + j < n_free ? __ldcg(list + at + j) : -1;
        if (id < 0) err |= DEVERR_NO_PAGES;
        else P.refs[(long long)s * P.num_blocks + id] = 1;
        to[have + j - split] = id;
      }
    }
  }
  err = __reduce_or_sync(0xffffffffu, err);
  if (err && lane == 0) flag_error(P.dev_error, err);
}

constexpr int FORK_PHASES = 5;

__global__ void __launch_bounds__(PLAN_THREADS, 1) fork_plan_kernel(const PagePlan P, int first, int last) {
  __shared__ int sm[33];
  allow_dependent_launch();  // the copies may launch; they wait for this grid to finish
  for (int phase = first; phase <= last; ++phase) {
    if (phase == 0) fork_init(P);
    else if (phase == 1) fork_mark(P);
    else if (phase == 2) fork_count(P, sm);
    else if (phase == 3) fork_rank(P, sm);
    else fork_assign(P, sm);
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

// The entries of one row segment that count: below the sequence's last token.
// Calls f(index in the table, entry or -1).
template <typename F>
__device__ __forceinline__ void compact_entries(const PagePlan& P, bool report, F f) {
  constexpr int SEG = 128;
  const int lane = threadIdx.x & 31;
  const int segs = (P.max_blocks + SEG - 1) / SEG;
  const long long tasks = (long long)P.batch * P.spaces * segs;
  const long long cap = (long long)P.max_blocks * P.block_size;
  int err = 0;
  for (long long t = (long long)blockIdx.x * (PLAN_THREADS / 32) + (threadIdx.x >> 5); t < tasks;
       t += (long long)gridDim.x * (PLAN_THREADS / 32)) {
    const long long r = t / segs;
    const int b = (int)(r / P.spaces), s = (int)(r % P.spaces), e0 = (int)(t % segs) * SEG;
    long long L = __ldg(P.seq_lens + b);
    if (L < 0) err |= DEVERR_SEQ_LEN;
    if (L > cap) err |= DEVERR_TABLE_RANGE;
    const int have = pages_of(P, (int)max(0LL, min(L, cap)));
    int v[SEG / 32];
#pragma unroll
    for (int k = 0; k < SEG / 32; ++k) {
      const int e = e0 + lane + 32 * k;
      v[k] = e < have ? __ldcg(P.table + r * P.max_blocks + e) : -1;
    }
#pragma unroll
    for (int k = 0; k < SEG / 32; ++k) {
      const int e = e0 + lane + 32 * k;
      if (v[k] >= P.num_blocks) err |= DEVERR_BLOCK_RANGE;
      if (e < P.max_blocks) f(r * P.max_blocks + e, s, v[k] < 0 || v[k] >= P.num_blocks ? -1 : v[k]);
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

__device__ __forceinline__ bool pinned(const PagePlan& P, long long u) { return P.pins && __ldg(P.pins + u) > 0; }

// Phase 2: used pages per task, and the used ones that may move.
__device__ void compact_count(const PagePlan& P, int* sm) {
  const int per_space = (P.num_blocks + UNITS_PER_TASK - 1) / UNITS_PER_TASK;
  const int tasks = P.spaces * per_space;
  for (int t = blockIdx.x; t < tasks; t += gridDim.x) {
    const int s = t / per_space, first = (t % per_space) * UNITS_PER_TASK + 4 * threadIdx.x;
    int used = 0, loose = 0, total;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long u = (long long)s * P.num_blocks + first + i;
      if (first + i < P.num_blocks && __ldcg(P.refs + u) > 0) {
        ++used;
        loose += !pinned(P, u);
      }
    }
    block_scan(used, sm, total);
    if (threadIdx.x == 0) P.task_count[t] = total;
    block_scan(loose, sm, total);
    if (threadIdx.x == 0) P.task_count[tasks + t] = total;
  }
}

// Phase 3: every page's rank: the holes and the movers listed in order, the
// map of all that stay.  row_ask / row_at hold the movers' count of each space.
__device__ void compact_rank(const PagePlan& P, int* sm) {
  const int per_space = (P.num_blocks + UNITS_PER_TASK - 1) / UNITS_PER_TASK;
  const int tasks = P.spaces * per_space;
  for (int t = blockIdx.x; t < tasks; t += gridDim.x) {
    const int s = t / per_space, k = t % per_space, first = k * UNITS_PER_TASK + 4 * threadIdx.x;
    const long long u0 = (long long)s * P.num_blocks;
    const int n_used = block_sum(P.task_count + s * per_space, per_space, sm);
    const int used_before = block_sum(P.task_count + s * per_space, k, sm);
    const int loose_before = block_sum(P.task_count + tasks + s * per_space, k, sm);
    // used pages below n_used that may move: whole tasks, then the rest one by one
    const int kb = n_used / UNITS_PER_TASK;
    int n = 0, below;
    for (int i = kb * UNITS_PER_TASK + threadIdx.x; i < n_used; i += PLAN_THREADS)
      n += __ldcg(P.refs + u0 + i) > 0 && !pinned(P, u0 + i);
    block_scan(n, sm, below);
    below += block_sum(P.task_count + tasks + s * per_space, kb, sm);
    bool used[4], loose[4];
    int nu = 0, nl = 0, total;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      used[i] = first + i < P.num_blocks && __ldcg(P.refs + u0 + first + i) > 0;
      loose[i] = used[i] && !pinned(P, u0 + first + i);
      nu += used[i];
      nl += loose[i];
    }
    int ru = used_before + block_scan(nu, sm, total);
    int rl = loose_before + block_scan(nl, sm, total) - below;
    if (k == per_space - 1 && threadIdx.x == 0) {
      P.num_used[s] = n_used;
      P.movers[s] = loose_before + total - below;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = first + i;
      if (id >= P.num_blocks) break;
      if (!used[i] && id < n_used && KVQ_IN_BOUNDS(ru <= id, P.dev_error))
        P.list[u0 + id - ru] = id;  // hole: as many holes before it as unused pages
      if (loose[i] && id >= n_used) {
        if (KVQ_IN_BOUNDS(rl >= 0 && rl < P.num_blocks, P.dev_error)) P.owner[u0 + rl] = id;  // mover
      } else {
        P.page_map[u0 + id] = used[i] ? id : -1;
      }
      ru += used[i];
      rl += loose[i];
    }
  }
}

// Phase 4: the movers' new numbers, their counts moved, the pairs to copy
// (the spaces' one after another).
__device__ void compact_pair(const PagePlan& P) {
  int before = 0;
  for (int s = 0; s < P.spaces; ++s) {
    const int n = __ldcg(P.movers + s);
    const long long u0 = (long long)s * P.num_blocks;
    for (long long k = (long long)blockIdx.x * PLAN_THREADS + threadIdx.x; k < n; k += (long long)gridDim.x * PLAN_THREADS) {
      const int src = __ldcg(P.owner + u0 + k), dst = __ldcg(P.list + u0 + k);
      if (!KVQ_IN_BOUNDS(dst >= 0 && dst < src && src < P.num_blocks && before + k < P.most_pairs, P.dev_error)) continue;
      P.page_map[u0 + src] = dst;
      P.refs[u0 + dst] = __ldcg(P.refs + u0 + src);
      P.refs[u0 + src] = 0;
      P.pair_src[before + k] = pool_unit(P, s, src);
      P.pair_dst[before + k] = pool_unit(P, s, dst);
    }
    before += n;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.num_pairs = before;
}

__device__ void compact_remap(const PagePlan& P) {
  compact_entries(P, false, [&](long long i, int s, int v) {
    P.new_table[i] = v >= 0 ? __ldcg(P.page_map + (long long)s * P.num_blocks + v) : -1;
  });
}

constexpr int COMPACT_PHASES = 6;

__global__ void __launch_bounds__(PLAN_THREADS, 1) compact_plan_kernel(const PagePlan P, int first, int last) {
  __shared__ int sm[33];
  allow_dependent_launch();  // the copies may launch; they wait for this grid to finish
  for (int phase = first; phase <= last; ++phase) {
    if (phase == 0) compact_init(P);
    else if (phase == 1) compact_mark(P);
    else if (phase == 2) compact_count(P, sm);
    else if (phase == 3) compact_rank(P, sm);
    else if (phase == 4) compact_pair(P);
    else compact_remap(P);
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

// One warp copies one piece (up to COPY_PIECE bytes) of one page of one pool
// at a time: eight 16-byte loads per lane in flight, then the stores.  A CTA
// takes a run of consecutive pieces of one pair.  How a pair is known to be
// free of conflicts: by construction (fork, compact), by the claims of the
// kernel before, or, for short lists, by the CTA itself, which compares the
// pair with the whole list (LISTED): that saves a launch, 6 of 221 us for 1200
// pages of 32 layers and 2 us of the host's time for a few pages.
constexpr int COPY_PIECE = 4096;
constexpr int COPY_RUN = 32;         // pieces per CTA and turn
constexpr int COPY_LISTED = 2048;    // pairs a CTA compares with
enum { COPY_SAFE, COPY_CLAIMED, COPY_CHECKS_LIST };

template <int CHECK>
__global__ void __launch_bounds__(256) copy_pages_kernel(const PageCopy P) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (CHECK != COPY_CHECKS_LIST) grid_dependency_wait();  // the pairs come from the kernel before
  const long long pairs = P.num_pairs_dev ? __ldcg(P.num_pairs_dev) : P.num_pairs;
  const int per_pair = 2 * P.num_layers * P.pieces, runs = (per_pair + P.run - 1) / P.run;
  for (long long w = blockIdx.x; w < pairs * runs; w += gridDim.x) {
    const long long i = w / runs;
    const int first = (int)(w % runs) * P.run;
    const int s = __ldcg(P.src + i), d = __ldcg(P.dst + i);
    if (s < 0 || d < 0 || s == d) continue;
    if (s >= P.units || d >= P.units) {
      if (first == 0 && threadIdx.x == 0) flag_error(P.dev_error, DEVERR_BLOCK_RANGE);
      continue;
    }
    bool conflict = false;  // read by another pair, or written by a lower one
    if (CHECK == COPY_CLAIMED) conflict = __ldcg(P.claim + d) != (int)i;
    if (CHECK == COPY_CHECKS_LIST) {
      int hit = 0;
      for (int j = threadIdx.x; j < P.num_pairs; j += 256) {
        const int a = __ldg(P.src + j), b = __ldg(P.dst + j);
        hit |= a >= 0 && b >= 0 && a < P.units && b < P.units && (a == d || (b == d && a != b && j < i));
      }
      conflict = __syncthreads_or(hit);
    }
    if (conflict) {
      if (first == 0 && threadIdx.x == 0) flag_error(P.dev_error, DEVERR_PAGE_CONFLICT);
      continue;
    }
    for (int item = first + warp; item < min(first + P.run, per_pair); item += 8) {
      const int lk = item / P.pieces, piece = item % P.pieces, layer = lk >> 1, bytes = P.unit_bytes[layer];
      const int size = ((bytes + P.pieces - 1) / P.pieces + 15) & ~15, lo = piece * size, n = min(size, bytes - lo);
      uint8_t* pool = (lk & 1) ? P.v[layer] : P.k[layer];
      const uint8_t* from = pool + (size_t)s * bytes + lo + 16 * lane;
      uint8_t* to = pool + (size_t)d * bytes + lo + 16 * lane;
      uint4 x[COPY_PIECE / 512];
#pragma unroll
      for (int k = 0; k < COPY_PIECE / 512; ++k)
        if (512 * k + 16 * lane < n) x[k] = *reinterpret_cast<const uint4*>(from + 512 * k);
#pragma unroll
      for (int k = 0; k < COPY_PIECE / 512; ++k)
        if (512 * k + 16 * lane < n) *reinterpret_cast<uint4*>(to + 512 * k) = x[k];
    }
  }
}

// ---------------------------------------------------------------------------
// launch

template <typename Kern, typename... Args>
cudaError_t launch_cluster(Kern kernel, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(PLAN_CLUSTER);
  cfg.blockDim = dim3(PLAN_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = PLAN_CLUSTER;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename Kern>
cudaError_t launch_plan(Kern kernel, const PagePlan& P, int phases, int sms, cudaStream_t stream) {
  const long long rows = (long long)(P.new_batch > P.batch ? P.new_batch : P.batch) * P.spaces;
  const long long work = (long long)P.spaces * P.num_blocks + rows * P.max_blocks;
  if (work <= PLAN_FUSED_WORK) return launch_cluster(kernel, stream, P, 0, phases - 1);
  for (int i = 0; i < phases; ++i) {
    kernel<<<sms, PLAN_THREADS, 0, stream>>>(P, i, i);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int CHECK>
cudaError_t launch_copies(PageCopy C, long long most_pairs, int sms, cudaStream_t stream) {
  int most = 0;
  for (int i = 0; i < C.num_layers; ++i) most = C.unit_bytes[i] > most ? C.unit_bytes[i] : most;
  C.pieces = (most + COPY_PIECE - 1) / COPY_PIECE;
  // long runs when there are pairs enough to fill the GPU with them, else one piece per warp
  const long long per_pair = 2LL * C.num_layers * C.pieces, resident = (long long)sms * 8;
  C.run = most_pairs * (per_pair / COPY_RUN) >= resident ? COPY_RUN : 8;
  const long long ctas = most_pairs * ((per_pair + C.run - 1) / C.run);
  if (ctas == 0) return cudaSuccess;
  const dim3 grid((unsigned)(ctas < resident ? ctas : resident));
  if (CHECK == COPY_CHECKS_LIST) {  // nothing before it to overlap with
    copy_pages_kernel<CHECK><<<grid, 256, 0, stream>>>(C);
    return cudaGetLastError();
  }
  return launch_dependent(copy_pages_kernel<CHECK>, grid, dim3(256), 0, stream, C);
}

}  // namespace

cudaError_t launch_copy_pages(const PageCopy& C, int sms, cudaStream_t stream) {
  if (C.num_pairs <= COPY_LISTED) return launch_copies<COPY_CHECKS_LIST>(C, C.num_pairs, sms, stream);
  const cudaError_t e = launch_cluster(copy_claim_kernel, stream, C);
  if (e != cudaSuccess) return e;
  return launch_copies<COPY_CLAIMED>(C, C.num_pairs, sms, stream);
}

cudaError_t launch_fork(const PagePlan& P, PageCopy C, int sms, cudaStream_t stream) {
  const cudaError_t e = launch_plan(fork_plan_kernel, P, FORK_PHASES, sms, stream);
  if (e != cudaSuccess) return e;
  C.src = P.pair_src;
  C.dst = P.pair_dst;
  C.num_pairs = P.new_batch * P.spaces;
  return launch_copies<COPY_SAFE>(C, C.num_pairs, sms, stream);
}

cudaError_t launch_compact(const PagePlan& P, PageCopy C, int sms, cudaStream_t stream) {
  const cudaError_t e = launch_plan(compact_plan_kernel, P, COMPACT_PHASES, sms, stream);
  if (e != cudaSuccess) return e;
  C.src = P.pair_src;
  C.dst = P.pair_dst;
  C.num_pairs_dev = P.num_pairs;
  return launch_copies<COPY_SAFE>(C, P.most_pairs, sms, stream);
}

}  // namespace kvq
