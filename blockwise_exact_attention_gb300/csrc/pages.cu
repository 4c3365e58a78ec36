// Pages that several requests of a cache share: forking a request, freeing one,
// moving the used pages to the lower end of the cache, and the copies that the
// first and the last ask for.
//
// shares[p] is the number of table rows that hold page p beyond the first, so a
// page that nobody shares has 0, as has a free one, and paged_plan hands out
// pages without touching it.
//
// Forking. One CTA checks the whole step, counts the pages that it needs (one for
// a fork that ends inside a page: that page is copied, so that no row ever adds
// tokens to a page that another one reads) and pops them in row order. Then a
// block per forked row copies the table's entries and counts them.
//
// Freeing. A block per ended row counts its pages down; then one cluster finds the
// pages nobody holds any more, those below 0, and pushes them in the order of
// their ids. Counting is by integer atomics, whose order does not matter: the same
// call gives the same stack.
//
// Compacting. The used pages go to the lowest ids: the lowest hole takes the
// highest used page, the next hole the next, as long as that is a move downwards.
// One CTA holds the pages as bits in shared memory, ranks holes from below and used
// pages from above, and lists the moves; the table is then mapped by the whole GPU.
//
// All of them are latency: some KB in a chain of dependent reads.
#include <cooperative_groups.h>

#include "launch_cache.cuh"
#include "pages.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace bea {
namespace {

namespace cg = cooperative_groups;

__device__ __forceinline__ int full_pages(int tokens, int page) { return tokens / page; }
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

// Block 0 does the step; the others copy the shares where they go to another array.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) fork_plan_kernel(const __grid_constant__ ForkParams p) {
  __shared__ int sums[kThreads / 32];
  grid_dependency_wait();
  if (blockIdx.x > 0) {
    copy_ints(p.s.shares_out, p.s.shares, p.s.num_pages, (int64_t)(blockIdx.x - 1) * kThreads + threadIdx.x,
              (int64_t)(gridDim.x - 1) * kThreads);
    return;
  }
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

__global__ void __launch_bounds__(kRowThreads) fork_rows_kernel(const __grid_constant__ ForkParams p) {
  grid_dependency_wait();
  for (int r = blockIdx.x; r < p.s.n; r += gridDim.x) {
    const int s = p.src[r], part = p.copies[3 * (int64_t)r + 2], len = p.s.lens_out[r];
    if (part < 0) continue;
    const int full = full_pages(len, p.s.page);
    const int32_t* from = p.table + s * p.table_stride;
    int32_t* to = p.table + r * p.table_stride;
    for (int c = threadIdx.x; c < full; c += kRowThreads) {
      const int id = from[c];
      to[c] = id;
      if (id >= 0 && id < p.s.num_pages)
        atomicAdd(p.s.shares_out + id, 1);
      else
        report_status(p.s.status, BEA_STATUS_PAGES);
    }
  }
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

__global__ void __launch_bounds__(kRowThreads) free_rows_kernel(const __grid_constant__ FreeParams p) {
  grid_dependency_wait();
  if (!height_fits(p.s, p.s.n_free[0])) return;
  for (int r = blockIdx.x; r < p.s.n; r += gridDim.x) {
    const int ends = p.ends[r], len = p.s.lens[r];
    if (ends >= 0 || !length_fits(p.s, len)) continue;
    const int held = pages_held(len, p.s.page);
    const int32_t* entries = p.table + r * p.table_stride;
    for (int c = threadIdx.x; c < held; c += kRowThreads) {
      const int id = entries[c];
      if (id >= 0 && id < p.s.num_pages)
        atomicSub(p.s.shares_out + id, 1);
      else
        report_status(p.s.status, BEA_STATUS_PAGES);
    }
  }
}

// One cluster, each CTA a run of the pages.
constexpr int kFreeThreads = 1024;
constexpr int kFreeCtas = 8;
constexpr int kFreeRun = 4;  // consecutive pages of a thread

__global__ void __cluster_dims__(kFreeCtas) __launch_bounds__(kFreeThreads)
    free_push_kernel(const __grid_constant__ FreeParams p) {
  __shared__ int sums[kFreeThreads / 32];
  __shared__ int counts[kFreeCtas];  // of every CTA's run
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  grid_dependency_wait();
  const int have = p.s.n_free[0];
  const bool ok = height_fits(p.s, have);
  constexpr int kTile = kFreeThreads * kFreeRun;
  // runs of whole tiles
  const int tiles = (p.s.num_pages + kTile - 1) / kTile, each = (tiles + kFreeCtas - 1) / kFreeCtas;
  const int64_t first = (int64_t)rank * each * kTile, last = min((int64_t)p.s.num_pages, first + (int64_t)each * kTile);
  int mine = 0;
  for (int64_t i = first + threadIdx.x; i < last; i += kFreeThreads) mine += p.s.shares_out[i] < 0;
  const int total = block_scan<kFreeThreads>(mine, sums).y;
  if (threadIdx.x < kFreeCtas) *cluster.map_shared_rank(&counts[rank], threadIdx.x) = total;
  cluster.sync();  // the counts are there, and the height and lengths below have not been written
  int at = have, all = 0;
  for (int c = 0; c < kFreeCtas; ++c) {
    if (c < rank) at += counts[c];
    all += counts[c];
  }
  bool lost = !ok;
  if (ok) {
    for (int64_t t0 = first; t0 < last; t0 += kTile) {
      const int64_t i0 = t0 + (int64_t)threadIdx.x * kFreeRun;
      int v[kFreeRun], n = 0;
#pragma unroll
      for (int z = 0; z < kFreeRun; ++z) {
        v[z] = i0 + z < last ? p.s.shares_out[i0 + z] : 0;
        n += v[z] < 0;
      }
      __syncthreads();  // `sums` is free
      const int2 s = block_scan<kFreeThreads>(n, sums);
      int to = at + s.x;
#pragma unroll
      for (int z = 0; z < kFreeRun; ++z) {
        if (v[z] >= 0) continue;
        if (to < p.s.n_pool)
          p.pool[to] = (int)(i0 + z);
        else
          lost = true;
        ++to;
        if (v[z] < -1) lost = true;  // more rows gave it back than held it
        p.s.shares_out[i0 + z] = 0;
      }
      at += s.y;
    }
  }
  if (rank == 0) {
    for (int r = threadIdx.x; r < p.s.n; r += kFreeThreads) {
      const int len = p.s.lens[r];
      const bool ends = p.ends[r] < 0;
      if (ends && !length_fits(p.s, len)) lost = true;
      p.s.lens_out[r] = ok && ends && length_fits(p.s, len) ? 0 : len;
    }
    if (threadIdx.x == 0) p.s.n_free_out[0] = ok ? min(have + all, p.s.n_pool) : have;
  }
  if (lost) report_status(p.s.status, BEA_STATUS_PAGES);
  cluster.sync();  // no CTA ends while another may still write its counts
}

// ---- compact ---------------------------------------------------------------------

// Every page to itself, no moves; the shares where they go to another array.
__global__ void __launch_bounds__(kRowThreads) compact_init_kernel(const __grid_constant__ CompactParams p) {
  grid_dependency_wait();
  const int64_t first = (int64_t)blockIdx.x * kRowThreads + threadIdx.x, step = (int64_t)gridDim.x * kRowThreads;
  for (int64_t i = first; i < p.s.num_pages; i += step) {
    p.page_map[i] = (int)i;
    if (p.s.shares_out != p.s.shares) p.s.shares_out[i] = p.s.shares[i];
  }
  for (int64_t i = first; i < 3 * (int64_t)p.capacity; i += step) p.copies[i] = -1;
}

constexpr int kCompactThreads = 1024;
__global__ void __launch_bounds__(kCompactThreads) compact_plan_kernel(const __grid_constant__ CompactParams p) {
  extern __shared__ uint32_t holes[];  // a bit per page: free
  __shared__ int sums[kCompactThreads / 32];
  const int pages = p.s.num_pages, words = (pages + 31) / 32, tid = threadIdx.x;
  for (int i = tid; i < words; i += kCompactThreads) holes[i] = 0u;
  __syncthreads();
  grid_dependency_wait();
  const int have = p.s.n_free[0];
  bool wrong = have < 0 || have > p.s.n_pool || have > pages;
  if (!wrong) {
    for (int i = tid; i < have; i += kCompactThreads) {
      const int id = p.pool[i];
      if (id < 0 || id >= pages) {
        wrong = true;
      } else if (atomicOr(&holes[id >> 5], 1u << (id & 31)) & (1u << (id & 31))) {
        wrong = true;  // twice on the stack
      }
    }
  }
  if (__syncthreads_or(wrong)) {
    if (tid == 0) report_status(p.s.status, BEA_STATUS_PAGES);
    if (p.pool_out != p.pool) copy_ints(p.pool_out, p.pool, p.s.n_pool, tid, kCompactThreads);
    return;
  }
  // Each thread has a run of words. Ranks of its first hole from below, of its first used page from below.
  const int per = (words + kCompactThreads - 1) / kCompactThreads;
  const int w0 = min(tid * per, words), w1 = min(w0 + per, words);
  int n = 0;
  for (int w = w0; w < w1; ++w) n += __popc(holes[w]);
  const int before = block_scan<kCompactThreads>(n, sums).x;
  const int used = pages - have;
  // moves: as many as there are holes below `used`
  int below = 0;
  for (int w = w0; w < w1 && w * 32 < used; ++w) {
    const int left = used - w * 32;
    below += __popc(left >= 32 ? holes[w] : holes[w] & ((1u << left) - 1u));
  }
  __syncthreads();
  const int moves = min(block_scan<kCompactThreads>(below, sums).y, p.capacity);
  int hole = before, taken = min(w0 * 32, pages) - before;
  for (int w = w0; w < w1; ++w) {
    const uint32_t here = w * 32 + 32 <= pages ? ~0u : (1u << (pages - w * 32)) - 1u;
    for (uint32_t b = holes[w]; b != 0 && hole < moves; b &= b - 1, ++hole) {
      p.copies[3 * (int64_t)hole + 1] = w * 32 + __ffs(b) - 1;
      p.copies[3 * (int64_t)hole + 2] = p.s.page;
    }
    const uint32_t free = holes[w];
    for (uint32_t b = ~free & here; b != 0; b &= b - 1, ++taken) {
      const int k = used - 1 - taken;  // rank from above
      if (k < moves) p.copies[3 * (int64_t)k] = w * 32 + __ffs(b) - 1;
    }
  }
  __syncthreads();
  for (int k = tid; k < moves; k += kCompactThreads) {
    const int from = p.copies[3 * (int64_t)k], to = p.copies[3 * (int64_t)k + 1];
    p.page_map[from] = to;
    p.s.shares_out[to] = p.s.shares[from];
    p.s.shares_out[from] = 0;
    atomicOr(&holes[from >> 5], 1u << (from & 31));
    atomicAnd(&holes[to >> 5], ~(1u << (to & 31)));
  }
  __syncthreads();
  // the new stack, the lowest page on top
  n = 0;
  for (int w = w0; w < w1; ++w) n += __popc(holes[w]);
  int at = have - 1 - block_scan<kCompactThreads>(n, sums).x;
  for (int w = w0; w < w1; ++w)
    for (uint32_t b = holes[w]; b != 0; b &= b - 1) p.pool_out[at--] = w * 32 + __ffs(b) - 1;
  for (int i = have + tid; i < p.s.n_pool; i += kCompactThreads) p.pool_out[i] = -1;
}

__global__ void __launch_bounds__(kRowThreads) compact_table_kernel(const __grid_constant__ CompactParams p) {
  grid_dependency_wait();
  for (int r = blockIdx.x; r < p.s.n; r += gridDim.x) {
    int len = p.s.lens[r];
    if (!length_fits(p.s, len)) {
      if (threadIdx.x == 0) report_status(p.s.status, BEA_STATUS_PAGES);
      len = len < 0 ? 0 : p.s.max_pages * p.s.page;
    }
    const int held = pages_held(len, p.s.page);
    const int32_t* from = p.table + r * p.table_stride;
    int32_t* to = p.table_out + r * p.table_out_stride;
    const int most = p.table_out == p.table ? held : p.s.max_pages;  // behind a row's pages its entries stay as they are
    for (int c = threadIdx.x; c < most; c += kRowThreads) {
      int id = from[c];
      if (c < held) {
        if (id >= 0 && id < p.s.num_pages)
          id = p.page_map[id];
        else
          report_status(p.s.status, BEA_STATUS_PAGES);
      }
      to[c] = id;
    }
  }
}

// ---- copy ------------------------------------------------------------------------

// HBM-bound: whole tokens of a page to another page, in every cache. A unit is (copy, cache, chunk of kChunk 16-byte
// pieces); which copies are there only the device knows, so one wave of blocks steps over the units, each looking 32 of
// its own ahead at once.
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

constexpr int kMostRowBlocks = 152 * 8;  // of kRowThreads: a wave

}  // namespace

cudaError_t launch_paged_fork(const ForkParams& p, cudaStream_t s, int* nlaunch) {
  const unsigned more = p.s.shares_out != p.s.shares ? grid_of(p.s.num_pages, 4096, 64) : 0;
  cudaError_t e = p.s.n <= 256 ? launch_dependent(fork_plan_kernel<256>, dim3(1 + more), 256, 0, s, p)
                               : launch_dependent(fork_plan_kernel<1024>, dim3(1 + more), 1024, 0, s, p);
  if (e != cudaSuccess) return e;
  *nlaunch += 1;
  if (p.s.n == 0) return e;
  e = launch_dependent(fork_rows_kernel, dim3(grid_of(p.s.n, 1, kMostRowBlocks)), kRowThreads, 0, s, p);
  if (e == cudaSuccess) *nlaunch += 1;
  return e;
}

cudaError_t launch_paged_free(const FreeParams& p, cudaStream_t s, int* nlaunch) {
  cudaError_t e;
  if (p.s.shares_out != p.s.shares && p.s.num_pages > 0) {
    e = launch_dependent(copy_shares_kernel, dim3(grid_of(p.s.num_pages, 1024, 152)), kRowThreads, 0, s, p.s);
    if (e != cudaSuccess) return e;
    *nlaunch += 1;
  }
  if (p.s.n > 0) {
    e = launch_dependent(free_rows_kernel, dim3(grid_of(p.s.n, 1, kMostRowBlocks)), kRowThreads, 0, s, p);
    if (e != cudaSuccess) return e;
    *nlaunch += 1;
  }
  e = launch_dependent(free_push_kernel, dim3(kFreeCtas), kFreeThreads, 0, s, p);
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
  const int64_t most = p.s.num_pages > 3 * (int64_t)p.capacity ? p.s.num_pages : 3 * (int64_t)p.capacity;
  if (most > 0) {
    e = launch_dependent(compact_init_kernel, dim3(grid_of(most, 1024, 152)), kRowThreads, 0, s, p);
    if (e != cudaSuccess) return e;
    *nlaunch += 1;
  }
  const size_t smem = ((size_t)p.s.num_pages + 31) / 32 * 4;
  e = launch_dependent(compact_plan_kernel, dim3(1), kCompactThreads, smem, s, p);
  if (e != cudaSuccess) return e;
  *nlaunch += 1;
  if (p.s.n == 0) return e;
  e = launch_dependent(compact_table_kernel, dim3(grid_of(p.s.n, 1, kMostRowBlocks)), kRowThreads, 0, s, p);
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
