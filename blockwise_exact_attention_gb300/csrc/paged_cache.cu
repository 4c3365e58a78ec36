// The paged cache's bookkeeping and its write: block tables, slot map and
// positions from request lengths, and new keys and values scattered to their
// slots.
//
// paged_plan. One CTA scans the requests (exclusive sums of pages given back,
// pages taken, tokens added), checks the whole step before it changes anything,
// pushes the pages of ended requests and writes the per-request arrays. The
// places of the added tokens are then independent of one another: token i of row
// r has position p = len_r + i and lives in page p / page of its row, which is
// either an old entry of the table or the page popped for it, pool[top - 1 -
// (cu_pages[r] + k)]. The token that opens a page also writes the table's entry,
// so no thread reads an entry that this step writes. Up to kFuseCapacity places
// the same CTA fills them row by row; above, a second launch spreads them over
// the GPU and finds their rows in cu_new.
//
// Latency-bound: a decode step moves some KB, in a chain of dependent reads
// (lengths, then table or stack) with a block-wide scan between them. A step of
// 256 requests takes 3.6 us of GPU time, one of 1024 requests that ends 50 of up
// to 16k tokens and adds 0.5 M tokens 13.1 us, more than half in the scanning CTA.
#include "launch_cache.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace bea {
namespace {

constexpr int kFillThreads = 256;
// Consecutive places of a thread: 16 bytes of each array, one search for the row. 0.5 M places of 1024 requests 13.2 us; 2:
// the same, 1: 15.0 us, 8: 14.6 us. (Below 20,000 places 1 is faster: 64 requests of 4000 5.0 against 6.7 us.)
constexpr int kFillRun = 4;
constexpr int kFillRows = 2048;  // up to as many rows' cu_new are searched in shared memory
// Up to this many places the scanning CTA fills them itself: 772 requests of a token each 6.2 us, 10.7 with the second
// launch; 64 requests and 1024 places 6.1 against 6.8 us, but 4000 places 7.5 against 6.6 us.
constexpr int kFuseCapacity = 2048;

__device__ __forceinline__ int pages_of(int tokens, int page) { return (int)(((int64_t)tokens + page - 1) / page); }

// Pages given back, pages taken, tokens added. A sum that reaches kMany stays there; no step is done with such a sum, and
// below it sums are exact.
constexpr uint32_t kMany = (1u << 31) - 1;
struct Sums {
  uint32_t back, need, add;
  __device__ __forceinline__ Sums operator+(const Sums& o) const {
    return {min(back + o.back, kMany), min(need + o.need, kMany), min(add + o.add, kMany)};
  }
};
__device__ __forceinline__ Sums warp_inclusive(Sums x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums y{__shfl_up_sync(~0u, x.back, o), __shfl_up_sync(~0u, x.need, o), __shfl_up_sync(~0u, x.add, o)};
    if ((threadIdx.x & 31) >= o) x = x + y;
  }
  return x;
}

// One row of the step.
struct Row {
  int len, add, back, had, need;
  bool wrong;
  __device__ __forceinline__ Sums sums() const { return {(uint32_t)back, (uint32_t)need, (uint32_t)add}; }
};
__device__ __forceinline__ Row row_of(const PlanParams& p, int len, int a) {
  Row r{len, 0, 0, 0, 0, false};
  if (len < 0 || a < -1 || (int64_t)len + max(a, 0) > (int64_t)p.max_pages * p.page) {
    r.wrong = true;
    return r;
  }
  r.had = pages_of(len, p.page);
  if (a < 0) {
    r.back = r.had;
  } else {
    r.add = a;
    r.need = pages_of(len + a, p.page) - r.had;
  }
  return r;
}

// The place of token i of a row that held `old` tokens: writes the slot, the position and, for a page's first token,
// the table's entry. `taken`: pages popped before the row.
__device__ __forceinline__ int2 place_of(const PlanParams& p, int row, int old, int i, int taken, int top) {
  const int pos = old + i, j = pos / p.page, off = pos - j * p.page, had = pages_of(old, p.page);
  int32_t* entry = p.table + row * p.table_stride + j;
  const int id = j < had ? *entry : p.pool[top - 1 - (taken + j - had)];
  if (off == 0) *entry = id;
  const int64_t at = (int64_t)id * p.page + off;
  if (id >= 0 && at <= INT32_MAX) return make_int2((int)at, pos);
  report_status(p.status, BEA_STATUS_PAGES);
  return make_int2(-1, pos);
}

// kPlanThreads: 256 for up to as many requests (a block of a quarter the size starts and meets sooner: 256 requests 4.0
// us, with 1024 threads 4.8 us), else 1024.
template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanParams p, int fill) {
  constexpr int kPlanWarps = kPlanThreads / 32;
  __shared__ Sums warp_sums[kPlanWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (fill) grid_launch_dependents();  // one CTA: the next kernel is set up beside it
  grid_dependency_wait();
  // 1. Totals and checks, before anything is changed. A thread has `per` consecutive rows.
  const int per = (p.n + kPlanThreads - 1) / kPlanThreads, r0 = tid * per;
  const int have = p.n_free[0];
  Sums mine{0, 0, 0};
  bool wrong = false;
  int len = 0, a = 0;  // of the thread's only row, where it has one
  for (int x = 0; x < per; ++x) {
    if (r0 + x >= p.n) break;
    len = p.lens[r0 + x];
    a = p.new_lens[r0 + x];
    const Row r = row_of(p, len, a);
    wrong = wrong || r.wrong;
    mine = mine + r.sums();
  }
  const Sums inc = warp_inclusive(mine);
  if (lane == 31) warp_sums[warp] = inc;
  const bool bad = __syncthreads_or(wrong);
  const Sums w = warp_inclusive(lane < kPlanWarps ? warp_sums[lane] : Sums{0, 0, 0});  // by every warp for itself
  const Sums all{__shfl_sync(~0u, w.back, 31), __shfl_sync(~0u, w.need, 31), __shfl_sync(~0u, w.add, 31)};
  const int prev = max(warp - 1, 0);
  Sums at{__shfl_sync(~0u, w.back, prev), __shfl_sync(~0u, w.need, prev), __shfl_sync(~0u, w.add, prev)};
  if (warp == 0) at = Sums{0, 0, 0};
  at = Sums{at.back + inc.back - mine.back, at.need + inc.need - mine.need, at.add + inc.add - mine.add};
  const int64_t top64 = (int64_t)have + all.back;
  const bool ok = !bad && have >= 0 && top64 <= p.n_pool && all.need <= top64 && all.add <= (uint32_t)p.capacity &&
                  max(all.back, max(all.need, all.add)) < kMany;
  const int top = (int)top64;
  if (!ok) {
    if (tid == 0) report_status(p.status, BEA_STATUS_PAGES);
    for (int r = tid; r <= p.n; r += kPlanThreads) {
      p.cu_new[r] = 0;
      p.cu_pages[r] = 0;
      if (r < p.n) p.lens_out[r] = p.lens[r];
    }
    __syncthreads();
    if (tid == 0) p.n_free_out[0] = have;
  } else {
    // 2. The arrays, and ended rows' pages onto the stack (by the whole warp, row after row).
    for (int x = 0; x < per; ++x) {
      const int row = r0 + x;
      Row r{0, 0, 0, 0, 0, false};
      if (row < p.n) {
        if (per > 1) len = p.lens[row], a = p.new_lens[row];
        r = row_of(p, len, a);
        p.cu_pages[row] = (int)at.need;
        p.cu_new[row] = (int)at.add;
        p.lens_out[row] = a < 0 ? 0 : len + a;
      }
      for (uint32_t ends = __ballot_sync(~0u, r.back > 0); ends != 0; ends &= ends - 1) {
        const int from = __ffs(ends) - 1;
        const int m = __shfl_sync(~0u, r.back, from), to = have + __shfl_sync(~0u, (int)at.back, from);
        const int32_t* entries = p.table + __shfl_sync(~0u, row, from) * p.table_stride;
        constexpr int kBatch = 16;
        for (int j = lane; j < m; j += 32 * kBatch) {
          int32_t id[kBatch];
#pragma unroll
          for (int z = 0; z < kBatch; ++z)
            if (j + 32 * z < m) id[z] = entries[j + 32 * z];
#pragma unroll
          for (int z = 0; z < kBatch; ++z)
            if (j + 32 * z < m) p.pool[to + j + 32 * z] = id[z];
        }
      }
      at = at + r.sums();
    }
    __syncthreads();  // the stack is complete, and n_free has been read by all (n_free_out may be the same word)
    if (tid == 0) {
      p.cu_pages[p.n] = (int)all.need;
      p.cu_new[p.n] = (int)all.add;
      p.n_free_out[0] = top - (int)all.need;
    }
  }
  if (!fill) return;
  // 3. The places, row after row: short rows by their thread, long ones by its warp.
  const int total = ok ? (int)all.add : 0;
  for (int i = total + tid; i < p.capacity; i += kPlanThreads) {
    p.slot_map[i] = -1;
    p.positions[i] = 0;
  }
  if (total == 0) return;
  // Tokens of a row that its thread places alone. 256 requests of one each 3.6 us, 1000 of up to two 6.4 us; 0: 18.4 and 25
  // us, 1: 3.5 and 9.3 us, 8: 3.6 and 6.4 us, but 64 requests of up to 64 6.1 instead of 5.8 us.
  constexpr int kShort = 2;
  at = Sums{at.back - mine.back, at.need - mine.need, at.add - mine.add};
  for (int x = 0; x < per; ++x) {
    const int row = r0 + x;
    Row r{0, 0, 0, 0, 0, false};
    int old = len;
    if (row < p.n) {
      if (per > 1) {  // the row's numbers as written above
        a = p.new_lens[row];
        old = p.lens_out[row] - a;
        at.add = (uint32_t)p.cu_new[row];
        at.need = (uint32_t)p.cu_pages[row];
      }
      r.add = max(a, 0);
    }
    if (r.add <= kShort)
      for (int i = 0; i < r.add; ++i) {
        const int2 s = place_of(p, row, old, i, (int)at.need, top);
        p.slot_map[at.add + i] = s.x;
        p.positions[at.add + i] = s.y;
      }
    for (uint32_t rows = __ballot_sync(~0u, r.add > kShort); rows != 0; rows &= rows - 1) {
      const int from = __ffs(rows) - 1;
      const int m = __shfl_sync(~0u, r.add, from), to = __shfl_sync(~0u, (int)at.add, from);
      const int w_row = __shfl_sync(~0u, row, from), w_old = __shfl_sync(~0u, old, from);
      const int w_taken = __shfl_sync(~0u, (int)at.need, from);
      for (int i = lane; i < m; i += 32) {
        const int2 s = place_of(p, w_row, w_old, i, w_taken, top);
        p.slot_map[to + i] = s.x;
        p.positions[to + i] = s.y;
      }
    }
  }
}

// The last row with cu[row] <= i among [lo, hi].
__device__ __forceinline__ int row_of_token(const int32_t* cu, int lo, int hi, int i) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= i)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kFillThreads) plan_fill_kernel(const __grid_constant__ PlanParams p) {
  grid_dependency_wait();
  constexpr int kWarpRun = 32 * kFillRun;
  __shared__ int32_t cu_shared[kFillRows + 1];
  const int lane = threadIdx.x & 31;
  const int32_t* cu = p.cu_new;  // searched: from shared memory where it fits
  if (p.n <= kFillRows) {
    for (int r = threadIdx.x; r <= p.n; r += kFillThreads) cu_shared[r] = p.cu_new[r];
    __syncthreads();
    cu = cu_shared;
  }
  const int total = cu[p.n], top = p.n_free_out[0] + p.cu_pages[p.n];
  const bool vec = ((reinterpret_cast<uintptr_t>(p.slot_map) | reinterpret_cast<uintptr_t>(p.positions)) & 15) == 0;
  const int64_t warps = (int64_t)gridDim.x * (kFillThreads / 32);
  for (int64_t w = (int64_t)blockIdx.x * (kFillThreads / 32) + (threadIdx.x >> 5); w * kWarpRun < p.capacity; w += warps) {
    const int first = (int)(w * kWarpRun), last = (int)min((int64_t)first + kWarpRun, (int64_t)total) - 1;
    // The rows of the warp's first and last token, by 32 probes at a time; each lane searches between them.
    int lo = 0, hi = 0;
    if (first < total) {
#pragma unroll
      for (int end = 0; end < 2; ++end) {
        const int i = end ? last : first;
        int x = end ? lo : 0, y = p.n - 1;  // the row is in [x, y]
        while (x < y) {
          const int step = (y - x + 32) / 32, at = x + step * lane;
          const uint32_t below = __ballot_sync(~0u, at <= y && cu[at] <= i);
          x += step * (31 - __clz(below));  // lane 0 is always below
          y = min(y, x + step - 1);
        }
        if (end == 0)
          lo = x;
        else
          hi = x;
      }
    }
    const int64_t i0 = (int64_t)first + lane * kFillRun;
    int32_t slot[kFillRun], pos[kFillRun];
    int row = i0 < total ? row_of_token(cu, lo, hi, (int)i0) : 0;
    int begin = 0, next = 0, old = 0, taken = 0;
    bool fresh = true;
#pragma unroll
    for (int z = 0; z < kFillRun; ++z) {
      slot[z] = -1;
      pos[z] = 0;
      if (i0 + z < total) {
        while (fresh || i0 + z >= next) {  // rows without tokens are passed over
          if (!fresh) ++row;
          fresh = false;
          begin = cu[row];
          next = cu[row + 1];
          old = p.lens_out[row] - (next - begin);
          taken = p.cu_pages[row];
        }
        const int2 s = place_of(p, row, old, (int)(i0 + z) - begin, taken, top);
        slot[z] = s.x;
        pos[z] = s.y;
      }
    }
    if (vec && i0 + kFillRun <= p.capacity) {
      *reinterpret_cast<int4*>(p.slot_map + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(p.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int z = 0; z < kFillRun; ++z)
        if (i0 + z < p.capacity) p.slot_map[i0 + z] = slot[z], p.positions[i0 + z] = pos[z];
    }
  }
}

// ---- write ---------------------------------------------------------------------

// HBM-bound copy of rows of some hundred bytes to places of their own: a thread
// moves 16 bytes of K and 16 of V. Index: of these pieces; 32 bits where they are
// enough, divisions by run-time numbers stand before every load (64,999 tokens of 8
// heads of 128 in bf16: 79.5 us, 6.7 TB/s; with 64-bit indexes 82.4 us; with four
// pieces a thread, loads first, 115 us). 251 such tokens take 1.5 us.
constexpr int kWriteThreads = 256;

template <typename Index>
__global__ void __launch_bounds__(kWriteThreads) paged_write_kernel(const __grid_constant__ PagedWriteParams p) {
  grid_dependency_wait();
  const unsigned per_token = p.hkv * p.row_vecs;
  const Index total = (Index)p.n * p.l * per_token;
  for (Index it = (Index)blockIdx.x * kWriteThreads + threadIdx.x; it < total; it += (Index)gridDim.x * kWriteThreads) {
    const Index t = it / per_token;
    const unsigned in = (unsigned)(it - t * per_token);
    const int slot = p.slot_map[t];
    const int64_t b = t / p.l;
    const int i = (int)(t - (Index)b * p.l);
    const int hh = in / p.row_vecs, c = in - hh * p.row_vecs;
    // read before the slot is known
    const uint4 kx = __ldcs(reinterpret_cast<const uint4*>(static_cast<const char*>(p.k.ptr) +
                                                           (b * p.k.sn + i * p.k.sl + hh * p.k.sh) * p.es + c * 16));
    const uint4 vx = __ldcs(reinterpret_cast<const uint4*>(static_cast<const char*>(p.v.ptr) +
                                                           (b * p.v.sn + i * p.v.sl + hh * p.v.sh) * p.es + c * 16));
    if (slot < 0 || slot >= p.num_slots) {
      if (slot != -1 && in == 0) report_status(p.status, BEA_STATUS_PAGES);
      continue;
    }
    const int pg = slot / p.page, off = slot - pg * p.page;
    const int64_t kd = (pg * p.k_cache.sn + off * p.k_cache.sl + hh * p.k_cache.sh) * p.es + c * 16;
    const int64_t vd = (pg * p.v_cache.sn + off * p.v_cache.sl + hh * p.v_cache.sh) * p.es + c * 16;
    *reinterpret_cast<uint4*>(static_cast<char*>(p.k_cache.ptr) + kd) = kx;
    *reinterpret_cast<uint4*>(static_cast<char*>(p.v_cache.ptr) + vd) = vx;
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanParams& p, cudaStream_t s, int* nlaunch) {
  const int fill = p.capacity <= kFuseCapacity;
  cudaError_t e = p.n <= 256 ? launch_dependent(plan_kernel<256>, dim3(1), 256, 0, s, p, fill)
                             : launch_dependent(plan_kernel<1024>, dim3(1), 1024, 0, s, p, fill);
  if (e != cudaSuccess) return e;
  *nlaunch += 1;
  if (fill) return cudaSuccess;
  static PerContext<int> cache;
  int cap = 0;
  if ((e = wave_cap(cache, plan_fill_kernel, kFillThreads, 0, &cap)) != cudaSuccess) return e;
  const int64_t blocks = ((int64_t)p.capacity + kFillThreads * kFillRun - 1) / (kFillThreads * kFillRun);
  e = launch_dependent(plan_fill_kernel, dim3((unsigned)(blocks < cap ? blocks : cap)), kFillThreads, 0, s, p);
  if (e == cudaSuccess) *nlaunch += 1;
  return e;
}

cudaError_t launch_paged_write(const PagedWriteParams& p, cudaStream_t s, int* nlaunch) {
  const int64_t total = (int64_t)p.n * p.l * p.hkv * p.row_vecs;
  if (total == 0) return cudaSuccess;
  int64_t blocks = (total + kWriteThreads - 1) / kWriteThreads;
  if (blocks > (int64_t(1) << 30)) blocks = int64_t(1) << 30;
  const bool narrow = blocks * kWriteThreads * 2 < (int64_t(1) << 32);
  const cudaError_t e = launch_dependent(narrow ? paged_write_kernel<uint32_t> : paged_write_kernel<uint64_t>,
                                         dim3((unsigned)blocks), kWriteThreads, 0, s, p);
  if (e == cudaSuccess) *nlaunch += 1;
  return e;
}

}  // namespace bea
