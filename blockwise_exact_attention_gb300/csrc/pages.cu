// Pages that several requests of a cache share: forking a request, freeing one,
// moving the used pages to the lower end of the cache, and the copies that the
// first and the last ask for.
//
// shares[p] is the number of table rows that hold page p beyond the first, so a
// page that nobody shares has 0, as has a free one, and paged_plan hands out
// pages without touching it.
//
// Forking. One block checks the whole step, counts the pages that it needs (one for
// a fork that ends inside a page: that page is copied, so that no row ever adds
// tokens to a page that another one reads) and pops them in row order. Then the
// forked rows' entries of the table are copied and counted.
//
// Freeing. The pages of the rows that end are counted down; then one cluster finds
// the pages nobody holds any more, those below 0, and pushes them in the order of
// their ids. Counting is by integer atomics, whose order does not matter: the same
// call gives the same stack.
//
// Compacting. The used pages go to the lowest ids: the lowest hole takes the
// highest used page, the next hole the next, as long as that is a move downwards.
// One block holds the pages as bits in shared memory, ranks holes from below and used
// pages from above, and lists the moves; then the table is mapped.
//
// All of them are latency: some KB in a chain of dependent reads. So one cluster of
// eight blocks does all of a call, with cluster barriers between its steps, where the
// table is small enough for eight SMs; above, each step is a launch over the GPU.
#include <cooperative_groups.h>

#include "launch_cache.cuh"
#include "pages.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace bea {
namespace {

namespace cg = cooperative_groups;

__device__ __forceinline__ int pages_held(int tokens, int page) { return tokens / page + (tokens % page != 0); }

// Sum of `x` over the threads before this one in the block, and over all of them. Every thread calls it; `sums` has a
// word per warp and is free again after the next barrier.
template <int kThreads>
__device__ __forceinline__ int2 block_scan(int x, int* sums) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  int w = lane < kWarps ? sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, w, o);
    if (lane >= o) w += y;
  }
  const int all = __shfl_sync(~0u, w, 31), prev = __shfl_sync(~0u, w, max(warp - 1, 0));
  return make_int2((warp == 0 ? 0 : prev) + inc - x, all);
}

__device__ __forceinline__ void copy_ints(int32_t* to, const int32_t* from, int n, int64_t first, int64_t step) {
  for (int64_t i = first; i < n; i += step) to[i] = from[i];
}

// ---- fork ------------------------------------------------------------------------

constexpr int kRowThreads = 256;
// Of the kernels that one cluster runs.
constexpr int kClusterThreads = 1024, kCtas = 8;

// The rows' entries dealt to a cluster's warps, several to a row where there are fewer rows than warps, as long as each has 64
// entries of a row's `width` (two rows of 8000 entries compacted by a warp each 87 us, so 8.5; a power of two: divisions took 0.5 us of a small fork's 6.5).
template <typename F>
__device__ __forceinline__ void rows_of_cluster(int n, int width, int rank, F f) {
  constexpr int kBits = 8;  // of a warp's number
  static_assert(kCtas * kClusterThreads / 32 == 1 << kBits, "the cluster's warps");
  const int warp = rank + kCtas * (threadIdx.x >> 5);
  const int row_bits = n > 1 ? 32 - __clz(n - 1) : 0, most = 31 - __clz(max((width + 63) / 64, 1));
  const int bits = max(0, min(kBits - row_bits, most));  // 2^bits warps to a row
  const int first = (warp & ((1 << bits) - 1)) * 32 + (threadIdx.x & 31);
  for (int r = warp >> bits; r < n; r += 1 << (kBits - bits)) f(r, first, 32 << bits);
}
// To a grid's blocks of kRowThreads, several to a row where there are fewer rows than blocks, as long as each has 1024 entries
// of a row's `width`.
template <typename F>
__device__ __forceinline__ void rows_of_grid(int n, int width, F f) {
  const int slices = max(1, min((int)gridDim.x / max(n, 1), (width + 1023) / 1024));
  for (int64_t i = blockIdx.x; i < (int64_t)n * slices; i += gridDim.x) {
    const int r = (int)(i / slices), slice = (int)(i - (int64_t)r * slices);
    f(r, slice * kRowThreads + (int)threadIdx.x, slices * kRowThreads);
  }
}

// One row of the step: how many tokens it takes (-1: it takes no part), and whether it is wrong.
struct ForkRow {
  int src, took;
  bool wrong;
};
__device__ __forceinline__ ForkRow fork_row(const ForkParams& p, int r) {
  const int s = p.src[r];
  if (s == -1) return {-1, -1, false};
  if (s < 0 || s >= p.s.n) return {s, -1, true};
  const int len = p.s.lens[s];
  int t = p.tokens != nullptr ? p.tokens[r] : -1;
  if (p.src[s] != -1 || p.s.lens[r] != 0 || len < 0 || len > (int64_t)p.s.max_pages * p.s.page || t < -1 || t > len)
    return {s, -1, true};
  return {s, t < 0 ? len : t, false};
}

// The step, by one block: checks, pops, and all of the outputs but the table's shared entries and their count.
template <int kThreads>
__device__ void fork_plan(const ForkParams& p, int* sums) {
  const int per = (p.s.n + kThreads - 1) / kThreads, r0 = threadIdx.x * per;
  const int have = p.s.n_free[0];
  int need = 0;
  bool wrong = false;
  for (int x = 0; x < per && r0 + x < p.s.n; ++x) {
    const ForkRow r = fork_row(p, r0 + x);
    wrong = wrong || r.wrong;
    need += r.took > 0 && r.took % p.s.page != 0;
  }
  const bool bad = __syncthreads_or(wrong);
  const int2 at = block_scan<kThreads>(need, sums);
  const bool ok = !bad && have >= 0 && have <= p.s.n_pool && at.y <= have;
  int top = have - at.x;
  for (int x = 0; x < per && r0 + x < p.s.n; ++x) {
    const int row = r0 + x;
    const ForkRow r = ok ? fork_row(p, row) : ForkRow{-1, -1, false};
    int from = -1, to = -1, part = r.took < 0 ? -1 : r.took % p.s.page;
    if (part > 0) {
      const int j = r.took / p.s.page;
      from = p.table[r.src * p.table_stride + j];
      to = p.pool[--top];
      p.table[row * p.table_stride + j] = to;
      if (from < 0 || from >= p.s.num_pages || to < 0 || to >= p.s.num_pages) {
        report_status(p.s.status, BEA_STATUS_PAGES);
        from = to = -1;
        part = 0;
      }
    }
    p.copies[3 * (int64_t)row] = from;
    p.copies[3 * (int64_t)row + 1] = to;
    p.copies[3 * (int64_t)row + 2] = part;
  }
  __syncthreads();  // lengths and height have been read by all: their outputs may be the same words
  // a row that forks was free, so no other row's length changes
  for (int x = 0; x < per && r0 + x < p.s.n; ++x) {
    const int row = r0 + x;
    int len = p.s.lens[row];
    if (ok && p.src[row] >= 0) {  // as fork_row, whose checks have passed; the source's length does not change
      const int t = p.tokens != nullptr ? p.tokens[row] : -1;
      len = t < 0 ? p.s.lens[p.src[row]] : t;
    }
    p.s.lens_out[row] = len;
  }
  if (threadIdx.x == 0) {
    p.s.n_free_out[0] = ok ? have - at.y : have;
    if (!ok) report_status(p.s.status, BEA_STATUS_PAGES);
  }
}

// The full pages of row r, by `step` threads of which this is the `first`-th.
__device__ __forceinline__ void fork_entries(const ForkParams& p, int r, int first, int step) {
  // (written by another SM in this launch, where one cluster does it all)
  const int s = p.src[r], part = __ldcg(p.copies + 3 * (int64_t)r + 2), len = __ldcg(p.s.lens_out + r);
  if (part < 0) return;
  const int full = len / p.s.page;
  const int32_t* from = p.table + s * p.table_stride;
  int32_t* to = p.table + r * p.table_stride;
#pragma unroll 4
  for (int c = first; c < full; c += step) {
    const int id = from[c];
    to[c] = id;
    if (id >= 0 && id < p.s.num_pages)
      atomicAdd(p.s.shares_out + id, 1);
    else
      report_status(p.s.status, BEA_STATUS_PAGES);
  }
}

// Block 0 does the step; the others copy the shares where they go to another array.
__global__ void __launch_bounds__(kClusterThreads) fork_plan_kernel(const __grid_constant__ ForkParams p) {
  __shared__ int sums[kClusterThreads / 32];
  grid_dependency_wait();
  if (blockIdx.x == 0)
    fork_plan<kClusterThreads>(p, sums);
  else
    copy_ints(p.s.shares_out, p.s.shares, p.s.num_pages, (int64_t)(blockIdx.x - 1) * kClusterThreads + threadIdx.x,
              (int64_t)(gridDim.x - 1) * kClusterThreads);
}
__global__ void __launch_bounds__(kRowThreads) fork_rows_kernel(const __grid_constant__ ForkParams p) {
  grid_dependency_wait();
  rows_of_grid(p.s.n, p.s.max_pages, [&](int r, int first, int step) { fork_entries(p, r, first, step); });
}

// All of it by one cluster: its first block the step, then its warps the rows.
__global__ void __cluster_dims__(kCtas) __launch_bounds__(kClusterThreads)
    fork_cluster_kernel(const __grid_constant__ ForkParams p) {
  __shared__ int sums[kClusterThreads / 32];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  grid_dependency_wait();
  if (rank == 0)
    fork_plan<kClusterThreads>(p, sums);
  else if (p.s.shares_out != p.s.shares)
    copy_ints(p.s.shares_out, p.s.shares, p.s.num_pages, (rank - 1) * kClusterThreads + (int)threadIdx.x,
              (kCtas - 1) * kClusterThreads);
  cluster.sync();
  rows_of_cluster(p.s.n, p.s.max_pages, rank, [&](int r, int first, int step) { fork_entries(p, r, first, step); });
}

// ---- free ------------------------------------------------------------------------

__global__ void __launch_bounds__(kRowThreads) copy_shares_kernel(const __grid_constant__ PagesState s) {
  grid_dependency_wait();
  copy_ints(s.shares_out, s.shares, s.num_pages, (int64_t)blockIdx.x * kRowThreads + threadIdx.x,
            (int64_t)gridDim.x * kRowThreads);
}

__device__ __forceinline__ bool height_fits(const PagesState& s, int have) { return have >= 0 && have <= s.n_pool; }
__device__ __forceinline__ bool length_fits(const PagesState& s, int len) {
  return len >= 0 && len <= (int64_t)s.max_pages * s.page;
}

// The pages of row r counted down if it ends, by `step` threads of which this is the `first`-th. (This thread's first entry is
// read beside the length and not behind it: an entry of a row that stays costs less than another latency.)
__device__ __forceinline__ void free_entries(const FreeParams& p, int r, int first, int step) {
  const int32_t* entries = p.table + r * p.table_stride;
  const int ends = p.ends[r], len = p.s.lens[r], entry = first < p.s.max_pages ? entries[first] : 0;
  if (ends >= 0 || !length_fits(p.s, len)) return;
  const int held = pages_held(len, p.s.page);
  auto give = [&](int id) {
    if (id >= 0 && id < p.s.num_pages)
      atomicSub(p.s.shares_out + id, 1);
    else
      report_status(p.s.status, BEA_STATUS_PAGES);
  };
  if (first < held) give(entry);
#pragma unroll 4
  for (int c = first + step; c < held; c += step) give(entries[c]);
}

__global__ void __launch_bounds__(kRowThreads) free_rows_kernel(const __grid_constant__ FreeParams p) {
  grid_dependency_wait();
  if (!height_fits(p.s, p.s.n_free[0])) return;
  rows_of_grid(p.s.n, p.s.max_pages, [&](int r, int first, int step) { free_entries(p, r, first, step); });
}

// One cluster, kTile pages at a time, read once: a warp takes kWords times 32 in a row, and lane j keeps a bit for each of the
// j-th 32 that nobody holds. kAll: the copy of the shares and the rows that end before it.
template <bool kAll>
__global__ void __cluster_dims__(kCtas) __launch_bounds__(kClusterThreads) free_push_kernel(const __grid_constant__ FreeParams p) {
  constexpr int kWords = 16, kTile = kCtas * kClusterThreads * kWords;
  __shared__ int sums[kClusterThreads / 32];
  __shared__ int counts[2][kCtas];  // of every CTA's run, of this tile and the next
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  grid_dependency_wait();
  const int have = p.s.n_free[0];
  const bool ok = height_fits(p.s, have);
  if constexpr (kAll) {
    if (p.s.shares_out != p.s.shares) {
      copy_ints(p.s.shares_out, p.s.shares, p.s.num_pages, rank * kClusterThreads + (int)threadIdx.x, kCtas * kClusterThreads);
      cluster.sync();
    }
    if (ok)
      rows_of_cluster(p.s.n, p.s.max_pages, rank, [&](int r, int first, int step) { free_entries(p, r, first, step); });
    cluster.sync();
  }
  int at = have;
  bool lost = !ok;
  // of a small cache fewer, so that all warps have some
  const int words = min(kWords, (p.s.num_pages + kCtas * kClusterThreads - 1) / (kCtas * kClusterThreads));
  const int lane = threadIdx.x & 31, warp = rank * (kClusterThreads / 32) + (threadIdx.x >> 5);
  int turn = 0;
  for (int64_t t0 = 0; t0 < p.s.num_pages; t0 += kTile, turn ^= 1) {
    const int64_t i0 = t0 + (int64_t)warp * words * 32;
    int v[kWords];
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      const int64_t id = i0 + j * 32 + lane;
      v[j] = j < words && id < p.s.num_pages ? __ldcg(p.s.shares_out + id) : 0;
    }
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      const uint32_t b = __ballot_sync(~0u, v[j] < 0);
      if (lane == j) mine = b;
      if (v[j] < -1) lost = true;  // more rows gave it back than held it
    }
    const int2 s = block_scan<kClusterThreads>(__popc(mine), sums);
    if (threadIdx.x < kCtas) *cluster.map_shared_rank(&counts[turn][rank], threadIdx.x) = s.y;
    cluster.sync();  // the counts are there, and what is written below has been read
    int to = at + s.x;
    for (int c = 0; c < kCtas; ++c) {
      if (c < rank) to += counts[turn][c];
      at += counts[turn][c];
    }
    if (!ok) continue;
    for (uint32_t some = __ballot_sync(~0u, mine != 0); some != 0; some &= some - 1) {
      const int j = __ffs(some) - 1;
      const uint32_t b = __shfl_sync(~0u, mine, j), bit = 1u << lane;
      const int where = __shfl_sync(~0u, to, j) + __popc(b & (bit - 1u));
      if (!(b & bit)) continue;
      const int64_t id = i0 + j * 32 + lane;
      if (where < p.s.n_pool)
        p.pool[where] = (int)id;
      else
        lost = true;
      p.s.shares_out[id] = 0;
    }
  }
  if (p.s.num_pages == 0) cluster.sync();  // the height and lengths have been read by all
  if (rank == 0) {
    for (int r = threadIdx.x; r < p.s.n; r += kClusterThreads) {
      const int len = p.s.lens[r];
      const bool ends = p.ends[r] < 0;
      if (ends && !length_fits(p.s, len)) lost = true;
      p.s.lens_out[r] = ok && ends && length_fits(p.s, len) ? 0 : len;
    }
    if (threadIdx.x == 0) p.s.n_free_out[0] = ok ? min(at, p.s.n_pool) : have;
  }
  if (lost) report_status(p.s.status, BEA_STATUS_PAGES);
  cluster.sync();  // no CTA ends while another may still write its counts
}

// ---- compact ---------------------------------------------------------------------

// Every page to itself, no moves; the shares where they go to another array.
__device__ __forceinline__ void compact_init(const CompactParams& p, int64_t first, int64_t step) {
  for (int64_t i = first; i < p.s.num_pages; i += step) {
    p.page_map[i] = (int)i;
    if (p.s.shares_out != p.s.shares) p.s.shares_out[i] = p.s.shares[i];
  }
  for (int64_t i = first; i < 3 * (int64_t)p.capacity; i += step) p.copies[i] = -1;
}

// 32 pages.
struct Word {
  int w;
  uint32_t taken, filled, left, free;  // bits of its pages: used before, holes to be filled, used ones that leave, free after
  int holes_at, taken_at, free_at;     // how many of these stand before it (taken: used before)
};

// The moves and the new stack, by one block, but for what compact_moves does. `wait` stands between what only reads and the
// first write to what compact_init writes. holes: a bit per page, zeros.
template <typename F>
__device__ void compact_plan(const CompactParams& p, uint32_t* holes, int* sums, F wait) {
  constexpr int kThreads = kClusterThreads;
  __shared__ Word todo[kThreads];
  const int pages = p.s.num_pages, words = (pages + 31) / 32, tid = threadIdx.x, lane = tid & 31;
  const int have = p.s.n_free[0];
  bool wrong = have < 0 || have > p.s.n_pool || have > pages;
  if (!wrong) {
#pragma unroll 8
    for (int i = tid; i < have; i += kThreads) {
      const int id = p.pool[i];
      if (id < 0 || id >= pages) {
        wrong = true;
      } else if (atomicOr(&holes[id >> 5], 1u << (id & 31)) & (1u << (id & 31))) {
        wrong = true;  // twice on the stack
      }
    }
  }
  if (__syncthreads_or(wrong)) {
    wait();
    if (tid == 0) report_status(p.s.status, BEA_STATUS_PAGES);
    if (p.pool_out != p.pool) copy_ints(p.pool_out, p.pool, p.s.n_pool, tid, kThreads);
    return;
  }
  // as many moves as there are holes below the place where the used pages end once all are moved
  const int used = pages - have;
  int below = 0;
  for (int w = tid; w * 32 < used; w += kThreads) {
    const int left = used - w * 32;
    below += __popc(left >= 32 ? holes[w] : holes[w] & ((1u << left) - 1u));
  }
  const int moves = min(block_scan<kThreads>(below, sums).y, p.capacity);
  wait();
  // Words in the order of the pages, a word per thread.
  int holes_before = 0, free_before = 0;  // in the words of earlier turns: holes, pages that are free in the end
  for (int w0 = 0; w0 < words; w0 += kThreads) {
    const int w = w0 + tid;
    const uint32_t here = w >= words ? 0u : w * 32 + 32 <= pages ? ~0u : (1u << (pages - w * 32)) - 1u;
    const uint32_t hole = w < words ? holes[w] : 0u, taken = ~hole & here;
    __syncthreads();  // `sums` is free
    const int2 h = block_scan<kThreads>(__popc(hole), sums);
    const int holes_at = holes_before + h.x;                       // holes before this word
    const int taken_at = min(w * 32, pages) - holes_at;            // used pages before it
    // the lowest `moves` holes are filled, the highest `moves` used pages leave
    uint32_t filled = 0u, left = 0u;
    const int fill = min(max(moves - holes_at, 0), 32), stay = min(max(used - moves - taken_at, 0), 32);
    if (fill >= __popc(hole)) {
      filled = hole;
    } else {
      uint32_t b = hole;
      for (int z = 0; z < fill; ++z) filled |= b & -b, b &= b - 1;
    }
    if (stay < __popc(taken)) {
      uint32_t b = taken;
      for (int z = 0; z < stay; ++z) b &= b - 1;
      left = b;
    }
    const uint32_t free = (hole & ~filled) | left;
    __syncthreads();
    const int2 f = block_scan<kThreads>(__popc(free), sums);
    const int free_at = free_before + f.x;
    holes_before += h.y;
    free_before += f.y;
    __syncthreads();
    // The words that have something to be written are dealt to the warps, whose lanes take a word's pages one each.
    const bool some = (filled | free) != 0u;
    const int2 q = block_scan<kThreads>(some, sums);
    if (some) todo[q.x] = Word{w, taken, filled, left, free, holes_at, taken_at, free_at};
    __syncthreads();
    for (int z = tid >> 5; z < q.y; z += kThreads / 32) {
      const Word d = todo[z];
      const int page = d.w * 32 + lane;
      const uint32_t mine = 1u << lane, lower = mine - 1u;
      if (d.filled & mine) {
        const int64_t k = 3 * (int64_t)(d.holes_at + __popc(d.filled & lower));  // all holes below a filled one are filled
        p.copies[k + 1] = page;
        p.copies[k + 2] = p.s.page;
      }
      if (d.left & mine) p.copies[3 * (int64_t)(used - 1 - (d.taken_at + __popc(d.taken & lower)))] = page;
      if (d.free & mine) p.pool_out[have - 1 - (d.free_at + __popc(d.free & lower))] = page;
    }
  }
  for (int i = have + tid; i < p.s.n_pool; i += kThreads) p.pool_out[i] = -1;
}

// What goes with the moves: the map of the pages and their owners.
__device__ __forceinline__ void compact_moves(const CompactParams& p, int64_t first, int64_t step) {
#pragma unroll 2
  for (int64_t k = first; k < p.capacity; k += step) {
    const int from = __ldcg(p.copies + 3 * k), to = __ldcg(p.copies + 3 * k + 1);
    if (from < 0) break;  // none behind the last
    p.page_map[from] = to;
    p.s.shares_out[to] = p.s.shares[from];
    p.s.shares_out[from] = 0;
  }
}

// Row r of the table, by `step` threads of which this is the `first`-th.
__device__ __forceinline__ void compact_entries(const CompactParams& p, int r, int first, int step) {
  int len = p.s.lens[r];
  if (!length_fits(p.s, len)) {
    if (first == 0) report_status(p.s.status, BEA_STATUS_PAGES);
    len = len < 0 ? 0 : p.s.max_pages * p.s.page;
  }
  const int held = pages_held(len, p.s.page);
  const int32_t* from = p.table + r * p.table_stride;
  int32_t* to = p.table_out + r * p.table_out_stride;
  const int most = p.table_out == p.table ? held : p.s.max_pages;  // behind a row's pages its entries stay as they are
#pragma unroll 4
  for (int c = first; c < most; c += step) {
    int id = from[c];
    if (c < held) {
      if (id >= 0 && id < p.s.num_pages)
        id = __ldcg(p.page_map + id);
      else
        report_status(p.s.status, BEA_STATUS_PAGES);
    }
    to[c] = id;
  }
}

__global__ void __launch_bounds__(kRowThreads) compact_init_kernel(const __grid_constant__ CompactParams p) {
  grid_dependency_wait();
  compact_init(p, (int64_t)blockIdx.x * kRowThreads + threadIdx.x, (int64_t)gridDim.x * kRowThreads);
}
__global__ void __launch_bounds__(kRowThreads) compact_moves_kernel(const __grid_constant__ CompactParams p) {
  grid_dependency_wait();
  compact_moves(p, (int64_t)blockIdx.x * kRowThreads + threadIdx.x, (int64_t)gridDim.x * kRowThreads);
}
__global__ void __launch_bounds__(kRowThreads) compact_table_kernel(const __grid_constant__ CompactParams p) {
  grid_dependency_wait();
  rows_of_grid(p.s.n, p.s.max_pages, [&](int r, int first, int step) { compact_entries(p, r, first, step); });
}

// One block, between the kernels above; or one cluster for everything, its first block for the plan.
__device__ __forceinline__ void clear_bits(const CompactParams& p, uint32_t* holes) {
  for (int i = threadIdx.x; i < (p.s.num_pages + 31) / 32; i += kClusterThreads) holes[i] = 0u;
  __syncthreads();
}
__global__ void __launch_bounds__(kClusterThreads) compact_plan_kernel(const __grid_constant__ CompactParams p) {
  extern __shared__ uint32_t holes[];
  __shared__ int sums[kClusterThreads / 32];
  clear_bits(p, holes);
  grid_dependency_wait();
  compact_plan(p, holes, sums, []() {});
}
__global__ void __cluster_dims__(kCtas) __launch_bounds__(kClusterThreads)
    compact_cluster_kernel(const __grid_constant__ CompactParams p) {
  extern __shared__ uint32_t holes[];
  __shared__ int sums[kClusterThreads / 32];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  if (rank == 0) clear_bits(p, holes);
  grid_dependency_wait();
  if (rank == 0) {
    compact_plan(p, holes, sums, [&]() { cluster.sync(); });
  } else {
    compact_init(p, (rank - 1) * kClusterThreads + (int)threadIdx.x, (kCtas - 1) * kClusterThreads);
    cluster.sync();
  }
  cluster.sync();  // the list of moves is there
  compact_moves(p, rank * kClusterThreads + (int)threadIdx.x, kCtas * kClusterThreads);
  cluster.sync();
  rows_of_cluster(p.s.n, p.s.max_pages, rank, [&](int r, int first, int step) { compact_entries(p, r, first, step); });
}

// ---- copy ------------------------------------------------------------------------

// HBM-bound: whole tokens of a page to another page, in every cache. A unit is (copy, cache, chunk of kChunk 16-byte
// pieces); which copies are there only the device knows, so one wave of blocks steps over the units, each looking 32 of
// its own ahead at once. 477 pages of 32 KB in four caches (125 MB moved) 17 us, the rate of a copy; the
// last pages of 200 forks, up to 64 KB in eight caches (96 MB) 16 us.
constexpr int kCopyThreads = 256;
constexpr int kCopyPieces = 4;  // of a thread at a time
constexpr int kChunk = kCopyThreads * kCopyPieces;

__global__ void __launch_bounds__(kCopyThreads) paged_copy_kernel(const __grid_constant__ CopyParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t units = (int64_t)p.m * p.n_caches * p.chunks;
  const unsigned per_copy = p.n_caches * p.chunks, per_token = p.hkv * p.row_vecs;
  grid_dependency_wait();
  for (int64_t u0 = blockIdx.x; u0 < units; u0 += (int64_t)gridDim.x * 32) {
    // lane z looks at the block's z-th unit from here
    const int64_t u = u0 + (int64_t)lane * gridDim.x;
    int from = -1, to = -1, todo = 0, where = 0;
    if (u < units) {
      const int64_t i = u / per_copy;
      where = (int)(u - i * per_copy);
      from = p.copies[3 * i];
      to = p.copies[3 * i + 1];
      const int tokens = p.copies[3 * i + 2];
      if (tokens > 0) {
        if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages || from == to || tokens > p.page) {
          if (where == 0 && threadIdx.x < 32) report_status(p.status, BEA_STATUS_PAGES);
        } else {
          todo = tokens * (int)per_token - where % p.chunks * kChunk;  // pieces of this chunk and those behind it
        }
      }
    }
    for (uint32_t live = __ballot_sync(~0u, todo > 0); live != 0; live &= live - 1) {
      const int z = __ffs(live) - 1;
      const int64_t f = __shfl_sync(~0u, from, z), t = __shfl_sync(~0u, to, z);
      const int left = __shfl_sync(~0u, todo, z), w = __shfl_sync(~0u, where, z);
      const int c = w / p.chunks, v0 = (w - c * p.chunks) * kChunk;
      const CopyParams::Cache& k = p.cache[c];
      const char* src = k.ptr + f * k.sn;
      char* dst = k.ptr + t * k.sn;
      uint4 x[kCopyPieces];
      int64_t at[kCopyPieces];
#pragma unroll
      for (int y = 0; y < kCopyPieces; ++y) {
        const int in = y * kCopyThreads + threadIdx.x, v = v0 + in;
        at[y] = (int64_t)v * 16;
        if (k.sl != 0) {
          const int tok = v / (int)per_token, rest = v - tok * (int)per_token, hh = rest / p.row_vecs;
          at[y] = tok * k.sl + hh * k.sh + (int64_t)(rest - hh * p.row_vecs) * 16;
        }
        if (in < left) x[y] = __ldcs(reinterpret_cast<const uint4*>(src + at[y]));
      }
#pragma unroll
      for (int y = 0; y < kCopyPieces; ++y)
        if (y * kCopyThreads + (int)threadIdx.x < left) __stcs(reinterpret_cast<uint4*>(dst + at[y]), x[y]);
    }
  }
}

unsigned grid_of(int64_t items, int64_t per, int most) {
  const int64_t b = (items + per - 1) / per;
  return (unsigned)(b < 1 ? 1 : b < most ? b : most);
}

// Blocks for the rows' entries.
unsigned row_blocks(const PagesState& s, int wave) { return grid_of(s.n * (((int64_t)s.max_pages + 1023) / 1024), 1, wave); }

// Blocks of kRowThreads: a wave of them, or one to an SM.
cudaError_t most_blocks(int* wave, int* each) {
  int sms = 0;
  const cudaError_t e = device_sm_count(&sms);
  *wave = sms * 8, *each = sms;
  return e;
}

}  // namespace

// Up to `entries` entries of a table and pages of a cache one cluster does all of a call, in one launch instead of two to four,
// each of which costs the host 1-2 us. In a graph, cluster and launches: 8 rows of 46 entries forked 4.4, 4.9 us, freed 5.8, 6.1, a
// cache of 242 pages compacted 7.3, 7.9 us; 64 rows of 128 entries 4.5, 4.9, 7.2, 8.0, 9.2, 10.5 us (4210 pages); 128 rows of 128
// (16384 entries) 4.6, 5.0, 7.2, 7.9, 10.5, 11.3 us; 256 rows of 128 (32768) 5.2, 5.1, 7.8, 8.0, 14.1, 13.7 us; 128 rows of 512
// 6.0, 5.2, 9.3, 8.7, 21.4, 19.1 us. Called one by one, 16384 entries: 6.0, 7.9, 7.5, 9.3, 10.4, 13.0 us; 32768: 5.9, 7.9, 7.9, 9.6,
// 14.2, 14.4 us.
static bool fits_cluster(const PagesState& s, int64_t entries) {
  return (int64_t)s.n * s.max_pages <= entries && s.num_pages <= entries;
}
constexpr int64_t kFewEntries = 16384, kFewCompacted = 32768;

cudaError_t launch_paged_fork(const ForkParams& p, cudaStream_t s, int* nlaunch) {
  cudaError_t e;
  if (fits_cluster(p.s, kFewEntries)) {
    e = launch_dependent(fork_cluster_kernel, dim3(kCtas), kClusterThreads, 0, s, p);
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
  }
  int wave = 0, each = 0;
  if ((e = most_blocks(&wave, &each)) != cudaSuccess) return e;
  const unsigned more = p.s.shares_out != p.s.shares ? grid_of(p.s.num_pages, 4096, each) : 0;
  if ((e = launch_dependent(fork_plan_kernel, dim3(1 + more), kClusterThreads, 0, s, p)) != cudaSuccess) return e;
  *nlaunch += 1;
  e = launch_dependent(fork_rows_kernel, dim3(row_blocks(p.s, wave)), kRowThreads, 0, s, p);
  if (e == cudaSuccess) *nlaunch += 1;
  return e;
}

cudaError_t launch_paged_free(const FreeParams& p, cudaStream_t s, int* nlaunch) {
  cudaError_t e;
  if (fits_cluster(p.s, kFewEntries)) {
    e = launch_dependent(free_push_kernel<true>, dim3(kCtas), kClusterThreads, 0, s, p);
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
  }
  int wave = 0, each = 0;
  if ((e = most_blocks(&wave, &each)) != cudaSuccess) return e;
  if (p.s.shares_out != p.s.shares) {
    e = launch_dependent(copy_shares_kernel, dim3(grid_of(p.s.num_pages, 1024, each)), kRowThreads, 0, s, p.s);
    if (e != cudaSuccess) return e;
    *nlaunch += 1;
  }
  e = launch_dependent(free_rows_kernel, dim3(row_blocks(p.s, wave)), kRowThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  *nlaunch += 1;
  e = launch_dependent(free_push_kernel<false>, dim3(kCtas), kClusterThreads, 0, s, p);
  if (e == cudaSuccess) *nlaunch += 1;
  return e;
}

cudaError_t launch_paged_compact(const CompactParams& p, cudaStream_t s, int* nlaunch) {
  static PerContext<int> cache;
  int done = 0;
  cudaError_t e = cache.get(
      [](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(compact_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kCompactMaxPages / 8);
      },
      &done);
  if (e != cudaSuccess) return e;
  const size_t smem = ((size_t)p.s.num_pages + 31) / 32 * 4;
  if (fits_cluster(p.s, kFewCompacted) && p.capacity <= kFewCompacted) {  // up to 4 KB of bits
    e = launch_dependent(compact_cluster_kernel, dim3(kCtas), kClusterThreads, smem, s, p);
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
  }
  int wave = 0, each = 0;
  if ((e = most_blocks(&wave, &each)) != cudaSuccess) return e;
  const int64_t most = p.s.num_pages > 3 * (int64_t)p.capacity ? p.s.num_pages : 3 * (int64_t)p.capacity;
  e = launch_dependent(compact_init_kernel, dim3(grid_of(most, 1024, each)), kRowThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  *nlaunch += 1;
  e = launch_dependent(compact_plan_kernel, dim3(1), kClusterThreads, smem, s, p);
  if (e != cudaSuccess) return e;
  *nlaunch += 1;
  e = launch_dependent(compact_moves_kernel, dim3(grid_of(p.capacity, 512, each)), kRowThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  *nlaunch += 1;
  e = launch_dependent(compact_table_kernel, dim3(row_blocks(p.s, wave)), kRowThreads, 0, s, p);
  if (e == cudaSuccess) *nlaunch += 1;
  return e;
}

int copy_chunks(int64_t page, int64_t hkv, int64_t row_vecs) { return (int)((page * hkv * row_vecs + kChunk - 1) / kChunk); }

cudaError_t launch_paged_copy(CopyParams& p, cudaStream_t s, int* nlaunch) {
  static PerContext<int> cache;
  int cap = 0;
  cudaError_t e = wave_cap(cache, paged_copy_kernel, kCopyThreads, 0, &cap);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)p.m * p.n_caches * p.chunks;
  e = launch_dependent(paged_copy_kernel, dim3(grid_of(units, 1, cap)), kCopyThreads, 0, s, p);
  if (e == cudaSuccess) *nlaunch += 1;
  return e;
}

}  // namespace bea
