// The paged cache's bookkeeping and its write: block tables, slot map and
// positions from request lengths, and new keys and values scattered to their
// slots.
//
// paged_plan. One CTA scans the requests (three exclusive sums: pages given
// back, pages taken, tokens added), checks the whole step before it changes
// anything, pushes the pages of ended requests and writes the per-request
// arrays. The places of the added tokens are then independent of one another:
// token i of row r (the row is found by bisection of cu_new) has position p =
// len_r + i and lives in page p / page of its row, which is either an old entry
// of the table or the page popped for it, pool[top - 1 - (cu_pages[r] + k)].
// The token that opens a page also writes the table's entry, so no thread reads
// an entry that this step writes.
#include "launch_cache.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace bea {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
// Up to this many places the scanning CTA fills them itself.
constexpr int kFuseCapacity = 4096;

__device__ __forceinline__ int pages_of(int tokens, int page) { return (int)(((int64_t)tokens + page - 1) / page); }

// Inclusive sum over the block of a pair of values; *total gets the block's sum.
__device__ __forceinline__ int2 block_scan(int2 x, int2* warp_sums, int2* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(~0u, x.x, o), b = __shfl_up_sync(~0u, x.y, o);
    if (lane >= o) x.x += a, x.y += b;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int2 w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(~0u, w.x, o), b = __shfl_up_sync(~0u, w.y, o);
      if (lane >= o) w.x += a, w.y += b;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  if (warp > 0) x.x += warp_sums[warp - 1].x, x.y += warp_sums[warp - 1].y;
  *total = warp_sums[31];
  __syncthreads();
  return x;
}

// Places [first, capacity) in steps of `stride`.
__device__ __forceinline__ void fill_places(const PlanParams& p, int64_t first, int64_t stride) {
  const int total = p.cu_new[p.n];
  const int top = p.n_free_out[0] + p.cu_pages[p.n];
  for (int64_t i = first; i < p.capacity; i += stride) {
    int slot = -1, pos = 0;
    if (i < total) {
      int lo = 0, hi = p.n - 1;  // the row with cu_new[row] <= i < cu_new[row + 1]
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_new[mid + 1] > i)
          hi = mid;
        else
          lo = mid + 1;
      }
      const int start = p.cu_new[lo];
      const int old = p.lens_out[lo] - (p.cu_new[lo + 1] - start);
      pos = old + (int)(i - start);
      const int j = pos / p.page, off = pos - j * p.page;
      const int had = pages_of(old, p.page);
      int32_t* entry = p.table + lo * p.table_stride + j;
      const int id = j < had ? *entry : p.pool[top - 1 - (p.cu_pages[lo] + j - had)];
      if (off == 0) *entry = id;
      const int64_t at = (int64_t)id * p.page + off;
      if (id >= 0 && at <= INT32_MAX)
        slot = (int)at;
      else
        report_status(p.status, BEA_STATUS_PAGES);
    }
    p.slot_map[i] = slot;
    p.positions[i] = pos;
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanParams p, int fill) {
  __shared__ int2 warp_sums[32];
  __shared__ long long sums[3];  // given back, taken, added
  __shared__ int bad;
  __shared__ int give_at[kPlanThreads], give_n[kPlanThreads];
  const int tid = threadIdx.x;
  if (tid < 3) sums[tid] = 0;
  if (tid == 0) bad = 0;
  grid_launch_dependents();
  __syncthreads();
  // 1. totals and checks, before anything is changed
  const int64_t most = (int64_t)p.max_pages * p.page;
  long long back = 0, need = 0, add = 0;
  bool wrong = false;
  for (int r = tid; r < p.n; r += kPlanThreads) {
    const int len = p.lens[r], a = p.new_lens[r];
    if (len < 0 || a < -1 || (int64_t)len + max(a, 0) > most) {
      wrong = true;
    } else if (a < 0) {
      back += pages_of(len, p.page);
    } else {
      need += pages_of(len + a, p.page) - pages_of(len, p.page);
      add += a;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    back += __shfl_xor_sync(~0u, back, o);
    need += __shfl_xor_sync(~0u, need, o);
    add += __shfl_xor_sync(~0u, add, o);
  }
  if ((tid & 31) == 0) {
    atomicAdd(reinterpret_cast<unsigned long long*>(&sums[0]), (unsigned long long)back);
    atomicAdd(reinterpret_cast<unsigned long long*>(&sums[1]), (unsigned long long)need);
    atomicAdd(reinterpret_cast<unsigned long long*>(&sums[2]), (unsigned long long)add);
  }
  if (wrong) bad = 1;
  __syncthreads();
  const int have = p.n_free[0];
  const bool ok = !bad && have >= 0 && have + sums[0] <= p.n_pool && sums[1] <= have + sums[0] && sums[2] <= p.capacity;
  __syncthreads();  // n_free has been read by all threads (n_free_out may be the same word)
  if (!ok) {
    if (tid == 0) report_status(p.status, BEA_STATUS_PAGES);
    for (int r = tid; r <= p.n; r += kPlanThreads) {
      p.cu_new[r] = 0;
      p.cu_pages[r] = 0;
      if (r < p.n) p.lens_out[r] = p.lens[r];
    }
    if (tid == 0) p.n_free_out[0] = have;
  } else {
    // 2. exclusive sums, 1024 rows at a time; ended rows' pages go on the stack
    int2 base = make_int2(0, 0);  // taken, added
    int given = 0;
    for (int r0 = 0; r0 < p.n; r0 += kPlanThreads) {
      const int r = r0 + tid;
      int len = 0, a = 0;
      if (r < p.n) len = p.lens[r], a = p.new_lens[r];
      const int ends = a < 0 ? pages_of(len, p.page) : 0;
      const int takes = a < 0 ? 0 : pages_of(len + a, p.page) - pages_of(len, p.page);
      const int adds = max(a, 0);
      int2 tot, tot_given;
      const int2 inc = block_scan(make_int2(takes, adds), warp_sums, &tot);
      const int2 inc_given = block_scan(make_int2(ends, 0), warp_sums, &tot_given);
      if (r < p.n) {
        p.cu_pages[r] = base.x + inc.x - takes;
        p.cu_new[r] = base.y + inc.y - adds;
        p.lens_out[r] = a < 0 ? 0 : len + a;
      }
      give_at[tid] = have + given + inc_given.x - ends;
      give_n[tid] = ends;
      base.x += tot.x;
      base.y += tot.y;
      given += tot_given.x;
      __syncthreads();
      if (tot_given.x > 0) {
        const int rows = min(kPlanThreads, p.n - r0);
        for (int w = tid >> 5; w < rows; w += kPlanThreads / 32) {
          const int m = give_n[w], at = give_at[w];
          const int32_t* row = p.table + (r0 + w) * p.table_stride;
          for (int j = tid & 31; j < m; j += 32) p.pool[at + j] = row[j];
        }
      }
      __syncthreads();
    }
    if (tid == 0) {
      p.cu_pages[p.n] = base.x;
      p.cu_new[p.n] = base.y;
      p.n_free_out[0] = have + given - base.x;
    }
  }
  if (fill) {
    __syncthreads();
    fill_places(p, tid, kPlanThreads);
  }
}

__global__ void __launch_bounds__(kFillThreads) plan_fill_kernel(PlanParams p) {
  grid_dependency_wait();
  fill_places(p, (int64_t)blockIdx.x * kFillThreads + threadIdx.x, (int64_t)gridDim.x * kFillThreads);
}

// ---- write ---------------------------------------------------------------------

constexpr int kWriteThreads = 256;

__global__ void __launch_bounds__(kWriteThreads) paged_write_kernel(const __grid_constant__ PagedWriteParams p) {
  const int per_token = p.hkv * p.row_vecs;
  const int64_t total = (int64_t)p.n * p.l * per_token;
  for (int64_t it = (int64_t)blockIdx.x * kWriteThreads + threadIdx.x; it < total;
       it += (int64_t)gridDim.x * kWriteThreads) {
    const int64_t t = it / per_token;
    const int in = (int)(it - t * per_token);
    const int hh = in / p.row_vecs, c = in - hh * p.row_vecs;
    const int slot = p.slot_map[t];
    if (slot < 0 || slot >= p.num_slots) {
      if (slot != -1 && in == 0) report_status(p.status, BEA_STATUS_PAGES);
      continue;
    }
    const int64_t b = t / p.l;
    const int i = (int)(t - b * p.l);
    const int pg = slot / p.page, off = slot - pg * p.page;
    const int64_t ks = (b * p.k.sn + i * p.k.sl + hh * p.k.sh) * p.es + c * 16;
    const int64_t vs = (b * p.v.sn + i * p.v.sl + hh * p.v.sh) * p.es + c * 16;
    const int64_t kd = (pg * p.k_cache.sn + off * p.k_cache.sl + hh * p.k_cache.sh) * p.es + c * 16;
    const int64_t vd = (pg * p.v_cache.sn + off * p.v_cache.sl + hh * p.v_cache.sh) * p.es + c * 16;
    const uint4 kx = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.k.ptr) + ks);
    const uint4 vx = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.v.ptr) + vs);
    *reinterpret_cast<uint4*>(static_cast<char*>(p.k_cache.ptr) + kd) = kx;
    *reinterpret_cast<uint4*>(static_cast<char*>(p.v_cache.ptr) + vd) = vx;
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanParams& p, cudaStream_t s, int* nlaunch) {
  const int fill = p.capacity <= kFuseCapacity;
  plan_kernel<<<1, kPlanThreads, 0, s>>>(p, fill);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  *nlaunch += 1;
  if (fill) return cudaSuccess;
  static PerContext<int> cache;
  int cap = 0;
  if ((e = wave_cap(cache, plan_fill_kernel, kFillThreads, 0, &cap)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int blocks = (p.capacity + kFillThreads - 1) / kFillThreads;
  cfg.gridDim = dim3((unsigned)(blocks < cap ? blocks : cap));
  cfg.blockDim = dim3(kFillThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, plan_fill_kernel, p);
  if (e != cudaSuccess) return e;
  *nlaunch += 1;
  return cudaSuccess;
}

cudaError_t launch_paged_write(const PagedWriteParams& p, cudaStream_t s, int* nlaunch) {
  const int64_t total = (int64_t)p.n * p.l * p.hkv * p.row_vecs;
  if (total == 0) return cudaSuccess;
  int64_t blocks = (total + kWriteThreads - 1) / kWriteThreads;
  if (blocks > (int64_t(1) << 30)) blocks = int64_t(1) << 30;
  paged_write_kernel<<<(unsigned)blocks, kWriteThreads, 0, s>>>(p);
  *nlaunch += 1;
  return cudaGetLastError();
}

}  // namespace bea
