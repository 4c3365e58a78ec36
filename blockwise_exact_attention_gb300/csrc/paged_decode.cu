// Attention of one new token per request over a paged K/V cache.
//
// out = sum_j p_j v_j / sum_j p_j with p_j = exp(scale q.k_j - m): one pass over
// the visible keys with a running maximum m and sum (online softmax), every key
// and value read once. HBM-bound: 2 d elements (K and V) a key and K/V head
// against 4 d g flops, g = h / h_kv query heads reading the same key. At 7 TB/s
// that is 28 TFLOP/s for g = 8 in bf16: too much for the CUDA cores beside the
// conversions, little for mma.sync with its 16 rows (112 TFLOP/s with the empty
// ones; with the weights in three terms the tensor pipe is a quarter and the issue
// slots a third busy). A tcgen05
// product has 64 rows at least, which 8 heads would leave empty, and its operands
// would have to meet in shared memory CTA-wide; here a warp goes through its keys
// alone. fp32 inputs stay exact: CUDA cores.
//
// Work. A UNIT is one (request, K/V head); its visible keys are cut into tiles of
// kKeys. The tiles of all units, request by request, make one list, and CTA c of
// G takes the c-th of G runs of it, each warp of the CTA an eighth of that. (With
// more than kRows query heads to a K/V head, neighbouring CTAs take the same run
// for kRows of them each, so that all but the first read from L2.) Nothing about
// the lengths is known on the host: every CTA finds its run from them, by a scan
// of tiles per request in shared memory. The runs cost the same, where a unit
// counts as its tiles and kUnitCost more for its queries and its output. A warp
// that covers a unit writes it; parts of a unit in several warps of a CTA are
// merged through shared memory when the warps are done, and parts in several CTAs
// go to the workspace as (O, m, l), which a second kernel joins in a fixed order
// (no atomics: the same call gives the same bits). If no unit is longer than
// kWholeTiles the CTAs' runs end at unit borders instead, and where the host sees
// that from the table's width it launches no second kernel.
//
// A warp streams its tiles by cp.async into a ring of its own, running ahead over
// unit borders, so no barrier stands before the end. Rows of a tile that no key
// of the request fills (behind its length, before its window, in a bad page)
// arrive as zeros and their scores are masked, so what those places hold in
// memory does not matter.
//
// Measured (GPU time, three sets of inputs in turn): 48 requests of 16k-32k keys,
// 32 / 8 heads of 128, bf16: 682-704 us, 6.8-7.1 TB/s (a copy reaches 6.8); one of
// 130k keys 83-85 us, 6.3-6.4 TB/s; 64 requests of 1-8192 keys 59-60 us, 5.7 TB/s:
// 2.5 us pass before the first load is sent (the lengths, their scan, the page
// table) and 5 at the end (the longest warp, the merge, the join); one request of
// 159 keys 5.7 us, all of it latency.
#include <algorithm>

#include <cuda_bf16.h>

#include "launch_cache.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace bea {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCtas = 160;       // one per SM
constexpr int kMaxRequests = 1024;  // per launch: their tile counts are scanned in shared memory
// Units up to this long are not cut between CTAs. 16: one request of 159 keys 8.3 instead of 7.3 us, 256 requests of
// 20-300 keys 39.8 instead of 37.1 us; 64: within 1% either way.
constexpr int kWholeTiles = 32;
// Of a unit, in tiles, besides its tiles. 1, 4, 6: within 1% on large batches, 4 and 6 2-5% slower on 73 requests of 32
// K/V heads.
constexpr int kUnitCost = 2;
// Of a CTA's run, as long as there are fewer than G such runs. 16, 32: one request of 159 keys 7.3, 9.6 instead of 5.4
// us.
constexpr int kMinCost = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Keys of a tile of rows of `d` elements (32, 64 or 128): K and V 4 KB each. (bf16, d = 64, with tiles of 16 keys, not
// 32: 66.0 against 68.6 us where pages of 16 tokens then hold a tile each, 82.6 against 64.7 us with pages of 20,
// whose rows are looked up one by one either way.)
__host__ __device__ constexpr int tile_keys(int d, bool is_f32) { return 4096 / (d * (is_f32 ? 4 : 2)); }

// kHd: query heads of a K/V head that a CTA takes at most (bf16: 8 or 16 of an mma's 16 rows).
template <bool kF32, int kD, int kHd>
struct Cfg {
  static constexpr int kRows = kHd;
  static constexpr int kEs = kF32 ? 4 : 2;
  static constexpr int kRowBytes = kD * kEs;
  static constexpr int kKeys = tile_keys(kD, kF32);  // of a tile
  static constexpr int kStageBytes = 2 * kKeys * kRowBytes;
  static constexpr int kPitch = kD + 8;  // floats a row of a part: 8 rows x 4 lanes fall on different banks
  static constexpr int kPart = kRows * kPitch * 4;
  static constexpr int kHeads = kWarps * kPart;  // a warp's first part; its last one takes its ring's place
  static constexpr int kQ = kF32 ? kWarps * kRows * kD * 4 : 0;
  static constexpr int kP = kF32 ? kWarps * kKeys * kRows * 4 : 0;
  // Tiles in a warp's ring. A third is slower (48 long requests 742 instead of 702 us, one of 130k keys 89.6 instead of
  // 85.1 us): the further the warps' streams run ahead, the less the memory sees of each row at a time.
  static constexpr int kStages = 2;
  static constexpr int kWarpRing = kStages * kStageBytes;
  static constexpr int kRing = kWarps * kWarpRing;
  static constexpr int kSmem = kRing + kHeads + kQ + kP;
  // The 16-byte pieces of row r are stored at piece ^ swizzle(r): the eight rows an ldmatrix reads (bf16), the two
  // rows by four pieces a quarter-warp reads (f32) fall on different banks.
  __host__ __device__ static constexpr int swizzle(int r) { return kF32 ? ((r & 1) << 2) | ((r & 7) >> 1) : r & 7; }
  static_assert(kKeys <= 32, "a tile's rows are bits of a mask");
  static_assert(kPart <= kWarpRing, "a part takes the place of its warp's ring");
};

// Workspace: [kMaxCtas] descriptors | [kMaxCtas][2][16] (m, l) | [kMaxCtas][2][rows][D] O. Entry 0 of a CTA is a
// unit that began before its run, entry 1 one that begins in the run and goes on after it.
struct Split {
  int b, hk, last, pad;  // last: the CTA that ends the unit; -1: nothing begins here that goes on
};
struct WsLayout {
  size_t ml, o, total;
};
__host__ __device__ inline WsLayout ws_layout(int rows, int d) {
  WsLayout w;
  w.ml = (size_t)kMaxCtas * sizeof(Split);
  w.o = w.ml + (size_t)kMaxCtas * 2 * 16 * 8;
  w.total = w.o + (size_t)kMaxCtas * 2 * rows * d * 4;
  return w;
}

// The part of a launch that is not in PagedDecodeParams.
struct Launch {
  int r0, n;     // requests [r0, r0 + n)
  int planes;    // blocks of kRows query heads per K/V head in this launch
  int head0;     // of a group, the first head of the first plane
  float sl2;     // scale * log2(e)
  int split;     // units may be cut: the workspace is there
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool read) {
  const int n = read ? 16 : 0;  // 0: the 16 bytes are set to zero and nothing is read
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The first 8 bits of a float, and two such as the bf16 numbers they are.
__device__ __forceinline__ float bf16_cut(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16x2_cut(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

// A row of kRows floats in shared memory, 16 bytes at a time where it can be.
template <int kRows>
__device__ __forceinline__ void store_rows(float* to, const float (&x)[kRows]) {
  if constexpr (kRows % 4 == 0) {
#pragma unroll
    for (int i = 0; i < kRows; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < kRows; ++i) to[i] = x[i];
  }
}
template <int kRows>
__device__ __forceinline__ void load_rows(const float* from, float (&x)[kRows]) {
  if constexpr (kRows % 4 == 0) {
#pragma unroll
    for (int i = 0; i < kRows; i += 4) {
      const float4 y = *reinterpret_cast<const float4*>(from + i);
      x[i] = y.x, x[i + 1] = y.y, x[i + 2] = y.z, x[i + 3] = y.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kRows; ++i) x[i] = from[i];
  }
}

// The first visible key of a request of `len` keys.
__device__ __forceinline__ int first_key(int len, int left) { return left >= len ? 0 : len - 1 - left; }

// m: in units of log2.
__device__ __forceinline__ void write_lse(const PagedDecodeParams& p, int64_t b, int hh, float m, float l) {
  p.lse.ptr[b * p.lse.sn + hh * p.lse.sh] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}
__device__ __forceinline__ void write_out4(const PagedDecodeParams& p, int64_t b, int hh, int c, float4 o, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t to = b * p.out.sn + hh * p.out.sh + c;
  o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (p.out_is_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(p.out.ptr) + to) = o;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out.ptr) + to) =
        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}

// The last index with key(index) <= x, key rising, key(0) <= x.
template <typename F>
__device__ __forceinline__ int last_below(int n, int x, F key) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (key(mid) <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// kSkip: requests' first keys are left out (another kernel's), p.skip of each.
template <bool kF32, int kD, int kHd, bool kSkip>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(const __grid_constant__ PagedDecodeParams p, const __grid_constant__ Launch a) {
  using C = Cfg<kF32, kD, kHd>;
  extern __shared__ __align__(128) uint8_t smem[];
  // requests with a visible key, in order: tiles of a unit summed over those before, number, length
  __shared__ int pre[kMaxRequests + 1], who[kMaxRequests], lens[kMaxRequests], skips[kSkip ? kMaxRequests : 1];
  __shared__ int4 warp_sums[kWarps];  // of a warp's requests: tiles, how many have some, the most
  __shared__ uint32_t masks[kWarps][C::kStages];
  __shared__ float2 ml[kWarps][2][16];  // of a warp's first and last part
  __shared__ int2 part_of[kWarps][2];   // (request, unit) of these parts, -1: none
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if constexpr (kSkip) {  // the kernel behind relies on what stands before this one being over (paged_shared.cu)
    grid_dependency_wait();
    grid_launch_dependents();
  } else {
    grid_launch_dependents();
    grid_dependency_wait();
  }

  // ---- tiles per request, their sums, and this CTA's run [t0, t1) -----------------
  // an empty cache has no page to read from: every length is past it
  const int most = p.num_pages > 0 ? p.max_pages * p.page : 0, units = p.hkv;
  // every plane has `grid` CTAs; cta: this one's place among its plane's
  const int grid = gridDim.x / a.planes, cta = blockIdx.x / a.planes, plane = blockIdx.x % a.planes;
  if (lane < 2) part_of[warp][lane] = make_int2(-1, -1);
  int run = 0, count = 0, longest = 0;
  for (int r0 = 0; r0 < a.n; r0 += kThreads) {
    const int r = r0 + tid;
    int len = r < a.n ? p.lens[a.r0 + r] : 0;
    if (len < 0 || len > most) {
      if (blockIdx.x == 0) report_status(p.status, BEA_STATUS_PAGES);
      len = len < 0 ? 0 : most;
    }
    const int skip = kSkip && r < a.n ? p.skip[a.r0 + r] : 0;
    const int begin = kSkip ? skip : first_key(len, p.left);
    const int tiles = len > begin ? (len + C::kKeys - 1) / C::kKeys - begin / C::kKeys : 0;
    const uint32_t some = __ballot_sync(~0u, tiles > 0);
    const int most_tiles = __reduce_max_sync(~0u, tiles);
    int inc = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) warp_sums[warp] = make_int4(inc, __popc(some), most_tiles, 0);
    __syncthreads();
    int at_tiles = run + inc - tiles, at = count + __popc(some & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int4 x = warp_sums[w];
      if (w < warp) at_tiles += x.x, at += x.y;
      run += x.x;
      count += x.y;
      longest = max(longest, x.z);
    }
    if (tiles > 0) {
      pre[at] = at_tiles;
      who[at] = a.r0 + r;
      lens[at] = len;
      if constexpr (kSkip) skips[at] = skip;
    }
    if (r0 + kThreads < a.n) __syncthreads();  // before warp_sums is written again
  }
  if (tid == 0) pre[count] = run;
  // requests without a visible key
  if (count < a.n) {
    for (int r = blockIdx.x; r < a.n; r += gridDim.x) {
      const int len = p.lens[a.r0 + r];
      if (min(len, most) > (kSkip ? p.skip[a.r0 + r] : 0)) continue;
      const int64_t b = a.r0 + r;
      for (int i = tid; i < p.h * p.d; i += kThreads) {
        const int hh = i / p.d;
        const int64_t to = b * p.out.sn + hh * p.out.sh + (i - hh * p.d);
        if (p.out_is_f32)
          static_cast<float*>(p.out.ptr)[to] = 0.f;
        else
          static_cast<__nv_bfloat16*>(p.out.ptr)[to] = __float2bfloat16(0.f);
      }
      for (int i = tid; i < p.h; i += kThreads) {
        p.lse.ptr[b * p.lse.sn + i * p.lse.sh] = -INFINITY;
        if constexpr (kSkip) p.cuts[b * p.h + i] = 0;
      }
    }
  }
  __syncthreads();

  // Costs (below 2^31, which the host sees to). Unit u of the k-th request costs its tiles and kUnitCost before them.
  const int cost = (run + kUnitCost * count) * units;
  const int ctas = min(grid, max(1, cost / kMinCost));
  const bool whole = longest <= kWholeTiles;
  const int share = cost / ctas, over = cost - share * ctas;  // the first `over` runs cost one more
  auto begin_cost = [&](int k) { return (pre[k] + kUnitCost * k) * units; };
  struct Place {
    int v, k, unit, in;  // a cost, its request and unit, and how far into the unit
  };
  auto place = [&](int v) {
    const int k = last_below(count, v, begin_cost);
    const int each = pre[k + 1] - pre[k] + kUnitCost, in = v - begin_cost(k), unit = in / each;
    return Place{v, k, unit, in - unit * each};
  };
  // where CTA c's run begins
  auto border = [&](int c) {
    int v = share * c + min(c, over);
    if (whole && v > 0 && v < cost) {
      const Place at = place(v);
      const int each = pre[at.k + 1] - pre[at.k] + kUnitCost;
      v += at.in * 2 < each ? -at.in : each - at.in;
    }
    return v;
  };
  // the first tile of the place's unit
  auto first_tile = [&](const Place& at) { return pre[at.k] * units + at.unit * (pre[at.k + 1] - pre[at.k]); };
  const WsLayout wl = ws_layout(C::kRows, kD);
  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  if (a.split && tid == 0) reinterpret_cast<Split*>(ws)[blockIdx.x] = Split{0, 0, -1, 0};  // until a unit is cut
  if (cta >= ctas || count == 0) return;
  // Searches and divisions side by side: lanes 0, 1 the CTA's run, then lanes 2, 3 this warp's eighth of it. (Of a
  // whole first unit the cost before its tiles is left out, so that no warp goes without tiles.)
  int mark = border(cta + (lane & 1));
  const int v0 = __shfl_sync(~0u, mark, 0), v1 = __shfl_sync(~0u, mark, 1);
  if (v0 >= v1) return;
  const int s0 = whole ? v0 + kUnitCost : v0;
  const int step = (v1 - s0) / kWarps, rest = v1 - s0 - step * kWarps, part_no = warp + (lane & 1);
  const int at_cost = (lane & 2) == 0 ? (lane == 0 ? v0 : v1) : s0 + step * part_no + min(part_no, rest);
  const Place at_place = place(min(at_cost, cost - 1));
  mark = at_cost >= cost ? run * units : first_tile(at_place) + max(0, at_place.in - kUnitCost);
  const int t0 = __shfl_sync(~0u, mark, 0), t1 = __shfl_sync(~0u, mark, 1);
  const int w0 = __shfl_sync(~0u, mark, 2), w1 = __shfl_sync(~0u, mark, 3);

  // ---- loads: the i-th tile of this warp is tile w0 + i -------------------------------
  auto tiles_before = [&](int k) { return pre[k] * units; };
  const uint32_t ring = smem_u32(smem) + warp * C::kWarpRing;
  const int group = p.h / p.hkv, head0 = a.head0 + plane * C::kRows, rows = min(C::kRows, group - head0);
  const int mine = w1 - w0;
  const bool one_page = p.page % C::kKeys == 0;  // a tile lies in one page
  auto page_of = [&](int key) { return p.page_shift >= 0 ? key >> p.page_shift : key / p.page; };
  // Descriptors of this warp's next 32 tiles, one per lane.
  int d_b = 0, d_hk = 0, d_key = 0;
  int64_t d_k = 0, d_v = 0;
  uint32_t d_mask = 0;
  auto describe = [&](int i) {
    d_mask = 0;
    d_k = d_v = 0;
    if (i >= mine) return;
    const int t = w0 + i;
    const int k = last_below(count, t, tiles_before);
    const int cnt = pre[k + 1] - pre[k], in = t - pre[k] * units, unit = in / cnt;
    const int len = lens[k], first = kSkip ? skips[k] : first_key(len, p.left);
    d_b = who[k];
    d_hk = unit;
    d_key = (first / C::kKeys + (in - unit * cnt)) * C::kKeys;
    // rows of the tile that are visible
    const int lo = max(first - d_key, 0), hi = min(len - d_key, C::kKeys);
    d_mask = (0xFFFFFFFFu >> (32 - hi)) & (0xFFFFFFFFu << lo);
    if (one_page) {
      const int pg = page_of(d_key), off = d_key - pg * p.page;
      const int id = p.table[d_b * p.table_stride + pg];
      if (id < 0 || id >= p.num_pages) {
        report_status(p.status, BEA_STATUS_PAGES);
        d_mask = 0;
      } else {
        d_k = (id * p.kc.sn + off * p.kc.sl + d_hk * p.kc.sh) * C::kEs;
        d_v = (id * p.vc.sn + off * p.vc.sl + d_hk * p.vc.sh) * C::kEs;
      }
    }
  };
  // Where tiles lie in several pages, lane r looks up the page of the tile's row r one tile ahead of its load.
  int n_id = -1, n_off = 0;
  auto look_up = [&](int i) {
    if (i >= mine) return;
    const int j = i & 31;
    if (j == 0) describe(i + lane);
    const int b = __shfl_sync(~0u, d_b, j), key = __shfl_sync(~0u, d_key, j) + lane;
    const uint32_t mask = __shfl_sync(~0u, d_mask, j);
    n_id = INT32_MIN;  // not visible
    if (lane < C::kKeys && ((mask >> lane) & 1u)) {
      const int pg = page_of(key);
      n_off = key - pg * p.page;
      n_id = max(p.table[b * p.table_stride + pg], -1);
    }
  };
  // This lane's 16-byte piece of a tile's rows sub, sub + kStep, ...
  constexpr int kChunks = kD * C::kEs / 16, kStep = 32 / kChunks;
  const int chunk = lane % kChunks, sub = lane / kChunks;
  const bool in_row = !kF32 || chunk * 4 < p.d;
  const int64_t k_lane = sub * p.kc.sl * C::kEs + chunk * 16, v_lane = sub * p.vc.sl * C::kEs + chunk * 16;
  const int64_t k_step = kStep * p.kc.sl * C::kEs, v_step = kStep * p.vc.sl * C::kEs;
  auto load = [&](int i) {
    if (i < mine) {
      const int j = i & 31, stage = i % C::kStages;
      if (!one_page && i == 0) look_up(0);
      const uint32_t kd = ring + stage * C::kStageBytes, vd = kd + C::kKeys * C::kRowBytes;
      uint32_t mask;
      int64_t k_at = 0, v_at = 0, k_row = 0, v_row = 0;
      if (one_page) {
        if (j == 0) describe(i + lane);
        mask = __shfl_sync(~0u, d_mask, j);
        k_at = __shfl_sync(~0u, d_k, j);
        v_at = __shfl_sync(~0u, d_v, j);
      } else {
        const int hk = __shfl_sync(~0u, d_hk, j);
        const bool ok = n_id >= 0 && n_id < p.num_pages;
        if (ok) {
          k_row = (n_id * p.kc.sn + n_off * p.kc.sl + hk * p.kc.sh) * C::kEs;
          v_row = (n_id * p.vc.sn + n_off * p.vc.sl + hk * p.vc.sh) * C::kEs;
        } else if (n_id != INT32_MIN) {
          report_status(p.status, BEA_STATUS_PAGES);
        }
        mask = __ballot_sync(~0u, ok);
      }
      if (lane == 0) masks[warp][stage] = mask;
      // A row that is not visible is not read: its address only has to be one (in the page, or in page 0).
#pragma unroll
      for (int it = 0; it < C::kKeys / kStep; ++it) {
        const int row = it * kStep + sub;
        const bool read = (mask >> row) & 1u;
        const uint32_t to = row * C::kRowBytes + ((chunk ^ C::swizzle(row)) << 4);
        int64_t ka = k_at + k_lane + it * k_step, va = v_at + v_lane + it * v_step;
        if (!one_page) ka = __shfl_sync(~0u, k_row, row) + chunk * 16, va = __shfl_sync(~0u, v_row, row) + chunk * 16;
        if (in_row) {
          cp_async16(kd + to, static_cast<const char*>(p.kc.ptr) + ka, read);
          cp_async16(vd + to, static_cast<const char*>(p.vc.ptr) + va, read);
        }
      }
      if (!one_page) look_up(i + 1);
    }
    cp_async_commit();  // an empty group where there is no tile, so that groups count tiles
  };

  // ---- unit by unit ----------------------------------------------------------------
  float* head = reinterpret_cast<float*>(smem + C::kRing + warp * C::kPart);
  float* tail = reinterpret_cast<float*>(smem + warp * C::kWarpRing);
  float* q_smem = reinterpret_cast<float*>(smem + C::kRing + C::kHeads) + warp * C::kRows * kD;
  float* p_smem = reinterpret_cast<float*>(smem + C::kRing + C::kHeads + C::kQ) + warp * C::kKeys * C::kRows;
  int done = 0, sent = 0;
  int k = __shfl_sync(~0u, at_place.k, 2), unit = __shfl_sync(~0u, at_place.unit, 2);
  while (done < mine) {
    const int cnt = pre[k + 1] - pre[k], begin = pre[k] * units + unit * cnt, end = begin + cnt;
    const int todo = min(end, w1) - w0;  // this warp's tiles up to the unit's end
    const int64_t b = who[k];
    const int h0 = unit * group + head0;
    const bool covered = begin >= w0 && end <= w1;
    const int which = begin < w0 ? 0 : 1;
    float* part = which == 0 ? head : tail;

    if constexpr (kF32) {
      // Scores: lane (key, quarter) takes every fourth 16-byte piece of its key's row.
      float m[C::kRows], l[C::kRows];  // l: this lane's keys only, quarter 0 counts
      float4 o[C::kRows];
#pragma unroll
      for (int i = 0; i < C::kRows; ++i) m[i] = -INFINITY, l[i] = 0.f, o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      const float* q = static_cast<const float*>(p.q.ptr) + b * p.q.sn + h0 * p.q.sh;
      __syncwarp();
      float4 qr[C::kRows];  // rows the unit does not have are zeros: computed along, never written
#pragma unroll
      for (int i = 0; i < C::kRows; ++i)
        qr[i] = i < rows && lane * 4 < p.d ? *reinterpret_cast<const float4*>(q + i * p.q.sh + lane * 4)
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < C::kRows; ++i)
        if (lane * 4 < kD) *reinterpret_cast<float4*>(q_smem + i * kD + lane * 4) = qr[i];
      __syncwarp();
      const int key = lane >> 2, quarter = lane & 3, sw = C::swizzle(key), pieces = p.d >> 2;
      constexpr int kCols = kD / 4, kParts = 32 / kCols;  // output: kParts lanes to 4 columns, each every kParts-th key
      const int col = lane % kCols, share_of = lane / kCols;
      for (; done < todo; ++done) {
        const int stage = done % C::kStages;
        while (sent < done + C::kStages) load(sent++);
        cp_async_wait<C::kStages - 1>();
        __syncwarp();
        const uint8_t* kt = smem + warp * C::kWarpRing + stage * C::kStageBytes;
        const uint8_t* vt = kt + C::kKeys * C::kRowBytes;
        const uint32_t mask = masks[warp][stage];
        constexpr int kGroups = C::kKeys / 8;  // keys key, key + 8, ... of this lane
        float s[kGroups][C::kRows];
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
          for (int i = 0; i < C::kRows; ++i) s[g][i] = 0.f;
#pragma unroll 2
        for (int c = quarter; c < pieces; c += 4) {
          float4 x[kGroups];
#pragma unroll
          for (int g = 0; g < kGroups; ++g)
            x[g] = *reinterpret_cast<const float4*>(kt + (key + 8 * g) * C::kRowBytes + ((c ^ sw) << 4));
#pragma unroll
          for (int i = 0; i < C::kRows; ++i) {
            const float4 y = *reinterpret_cast<const float4*>(q_smem + i * kD + c * 4);
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
              s[g][i] = fmaf(x[g].x, y.x, fmaf(x[g].y, y.y, fmaf(x[g].z, y.z, fmaf(x[g].w, y.w, s[g][i]))));
          }
        }
#pragma unroll
        for (int i = 0; i < C::kRows; ++i) {
          float top = -INFINITY;
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            s[g][i] += __shfl_xor_sync(~0u, s[g][i], 1);
            s[g][i] += __shfl_xor_sync(~0u, s[g][i], 2);
            s[g][i] = (mask >> (key + 8 * g)) & 1u ? s[g][i] * a.sl2 : -INFINITY;
            top = fmaxf(top, s[g][i]);
          }
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
          const float mn = fmaxf(m[i], top), w = mn == -INFINITY ? 1.f : ex2_approx(m[i] - mn);
          m[i] = mn;
          l[i] *= w;
          o[i] = make_float4(o[i].x * w, o[i].y * w, o[i].z * w, o[i].w * w);
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            s[g][i] = ex2_approx(s[g][i] - (mn == -INFINITY ? 0.f : mn));
            if (quarter == 0) l[i] += s[g][i];
          }
        }
        if (quarter == 0) {
#pragma unroll
          for (int g = 0; g < kGroups; ++g) store_rows<C::kRows>(p_smem + (key + 8 * g) * C::kRows, s[g]);
        }
        __syncwarp();
#pragma unroll
        for (int jj = 0; jj < C::kKeys / kParts; ++jj) {
          const int j = jj * kParts + share_of;
          const float4 v = *reinterpret_cast<const float4*>(vt + j * C::kRowBytes + ((col ^ C::swizzle(j)) << 4));
          float e[C::kRows];
          load_rows<C::kRows>(p_smem + j * C::kRows, e);
#pragma unroll
          for (int i = 0; i < C::kRows; ++i)
            o[i] = make_float4(fmaf(e[i], v.x, o[i].x), fmaf(e[i], v.y, o[i].y), fmaf(e[i], v.z, o[i].z),
                               fmaf(e[i], v.w, o[i].w));
        }
        __syncwarp();
      }
#pragma unroll
      for (int off = kCols; off < 32; off *= 2)
#pragma unroll
        for (int i = 0; i < C::kRows; ++i) {
          o[i].x += __shfl_xor_sync(~0u, o[i].x, off);
          o[i].y += __shfl_xor_sync(~0u, o[i].y, off);
          o[i].z += __shfl_xor_sync(~0u, o[i].z, off);
          o[i].w += __shfl_xor_sync(~0u, o[i].w, off);
        }
#pragma unroll
      for (int i = 0; i < C::kRows; ++i) {
        l[i] += __shfl_xor_sync(~0u, l[i], 4);
        l[i] += __shfl_xor_sync(~0u, l[i], 8);
        l[i] += __shfl_xor_sync(~0u, l[i], 16);
        l[i] = __shfl_sync(~0u, l[i], 0);
      }
      if (covered) {
#pragma unroll
        for (int i = 0; i < C::kRows; ++i) {
          if (i >= rows) break;
          const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
          if (lane * 4 < p.d)
            *reinterpret_cast<float4*>(static_cast<float*>(p.out.ptr) + b * p.out.sn + (h0 + i) * p.out.sh + lane * 4) =
                make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv);
          if (lane == 0) write_lse(p, b, h0 + i, m[i], l[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < C::kRows; ++i) {
          if (lane == 0) ml[warp][which][i] = make_float2(m[i], l[i]);
          if (lane * 4 < p.d) *reinterpret_cast<float4*>(part + i * C::kPitch + lane * 4) = o[i];
        }
      }
    } else {
      // m16n8k16: rows are query heads, S = Q K^T leaves P in the layout the second product takes as its A operand.
      float o[kD / 8][4];
#pragma unroll
      for (int i = 0; i < kD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      // rows 8-15 of the products stay empty where a unit has at most 8 heads
      constexpr int kHalves = C::kRows > 8 ? 2 : 1;
      float m[kHalves], l[kHalves];
#pragma unroll
      for (int x = 0; x < kHalves; ++x) m[x] = -INFINITY, l[x] = 0.f;
      const int row = lane >> 2, col = (lane & 3) * 2;
      uint32_t qf[kD / 16][4];
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q.ptr) + b * p.q.sn + h0 * p.q.sh;
#pragma unroll
      for (int ks = 0; ks < kD / 16; ++ks)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int i = row + (x & 1) * 8, c = ks * 16 + (x >> 1) * 8 + col;
          qf[ks][x] = (x & 1) < kHalves && i < rows ? *reinterpret_cast<const uint32_t*>(q + i * p.q.sh + c) : 0u;
        }
      for (; done < todo; ++done) {
        const int stage = done % C::kStages;
        while (sent < done + C::kStages) load(sent++);
        cp_async_wait<C::kStages - 1>();
        __syncwarp();
        const uint32_t kt = ring + stage * C::kStageBytes, vt = kt + C::kKeys * C::kRowBytes;
        const uint32_t mask = masks[warp][stage];
        constexpr int kSub = C::kKeys / 16;  // blocks of 16 keys
        float s[2 * kSub][4] = {};
#pragma unroll
        for (int ks = 0; ks < kD / 16; ++ks) {
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            uint32_t kf[4];
            const int kr = u * 16 + (lane & 7) + ((lane >> 4) << 3), chunk = 2 * ks + ((lane >> 3) & 1);
            ldsm4(kt + kr * C::kRowBytes + ((chunk ^ C::swizzle(kr)) << 4), kf);
            mma_bf16(s[2 * u], qf[ks], kf[0], kf[1]);
            mma_bf16(s[2 * u + 1], qf[ks], kf[2], kf[3]);
          }
        }
        if (mask != (0xFFFFFFFFu >> (32 - C::kKeys))) {
#pragma unroll
          for (int nb = 0; nb < 2 * kSub; ++nb)
#pragma unroll
            for (int x = 0; x < 2 * kHalves; ++x)
              if (!((mask >> (nb * 8 + col + (x & 1))) & 1u)) s[nb][x] = -INFINITY;
        }
        float top[kHalves];  // in units of log2, like m
#pragma unroll
        for (int x = 0; x < kHalves; ++x) {
          top[x] = fmaxf(s[0][2 * x], s[0][2 * x + 1]);
#pragma unroll
          for (int nb = 1; nb < 2 * kSub; ++nb) top[x] = fmax3(top[x], s[nb][2 * x], s[nb][2 * x + 1]);
          top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 1));
          top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 2)) * a.sl2;
        }
        // O and l are rescaled only when a maximum grows by more than 2^8: the reference value then in use
        // cancels in the end, and P stays below 2^8.
        bool grown = top[0] > m[0] + 8.f;
        if constexpr (kHalves == 2) grown = grown || top[1] > m[1] + 8.f;
        if (__any_sync(~0u, grown)) {
#pragma unroll
          for (int x = 0; x < kHalves; ++x) {
            const float mn = fmaxf(m[x], top[x]);
            const float w = mn == -INFINITY ? 1.f : ex2_approx(m[x] - mn);
            m[x] = mn;
            l[x] *= w;
#pragma unroll
            for (int i = 0; i < kD / 8; ++i) o[i][2 * x] *= w, o[i][2 * x + 1] *= w;
          }
        }
        // P as three bf16 terms of 8 bits each: all 24 of it, so that the product with V loses nothing of the weights.
        // The last two are kept above 0 (by 2^-24 of P at most), so that an infinite value stays infinite.
        uint32_t hi[kSub][4] = {}, mid[kSub][4] = {}, lo[kSub][4] = {};
#pragma unroll
        for (int x = 0; x < kHalves; ++x) {
          const float ref = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
          for (int nb = 0; nb < 2 * kSub; ++nb) {
            const float p0 = ex2_approx(fmaf(s[nb][2 * x], a.sl2, -ref)), p1 = ex2_approx(fmaf(s[nb][2 * x + 1], a.sl2, -ref));
            l[x] += p0 + p1;
            const float least0 = p0 * 0x1p-24f, least1 = p1 * 0x1p-24f;
            const float r0 = fmaxf(p0 - bf16_cut(p0), least0), r1 = fmaxf(p1 - bf16_cut(p1), least1);
            const float t0 = fmaxf(r0 - bf16_cut(r0), least0), t1 = fmaxf(r1 - bf16_cut(r1), least1);
            hi[nb / 2][(nb & 1) * 2 + x] = pack_bf16x2_cut(p0, p1);
            mid[nb / 2][(nb & 1) * 2 + x] = pack_bf16x2_cut(r0, r1);
            lo[nb / 2][(nb & 1) * 2 + x] = pack_bf16x2_cut(t0, t1);
          }
        }
        // A tile's products are summed from 0, small terms first, and added to O in fp32: the tensor core cuts its sums
        // off, which in one accumulator over all keys draws O towards 0 (48 requests of 16k-32k keys: fp32 output off by
        // 2.5e-5 of its size, so by 4.5e-7, and by 3.3e-6 and 2.7e-7 for one of 130k keys). With up to 8 heads the middle
        // terms take the rows 8-15 of the small terms' product, which no head has: 5% of the time where pages end inside
        // a tile, else within 1% of two terms in one accumulator; three products instead were 1-7%, 15% there. With 16
        // heads a product for each term: 1%, but 24% where two CTAs share a K/V head (97 -> 121 us) and a warp's own chain
        // of products is the bound (no wait for memory, the tensor pipe 38% busy).
#pragma unroll
        for (int dp = 0; dp < kD / 16; ++dp) {
          uint32_t vf[kSub][4];
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            const int vr = u * 16 + (lane & 7) + (((lane >> 3) & 1) << 3), chunk = 2 * dp + (lane >> 4);
            ldsm4_t(vt + vr * C::kRowBytes + ((chunk ^ C::swizzle(vr)) << 4), vf[u]);
          }
          float sum[2][4] = {};
          if constexpr (kHalves == 2) {
#pragma unroll
            for (int term = 0; term < 3; ++term)
#pragma unroll
              for (int u = 0; u < kSub; ++u) {
                const uint32_t(&w)[4] = term == 0 ? lo[u] : term == 1 ? mid[u] : hi[u];
                mma_bf16(sum[0], w, vf[u][0], vf[u][1]);
                mma_bf16(sum[1], w, vf[u][2], vf[u][3]);
              }
#pragma unroll
            for (int x = 0; x < 4; ++x) o[2 * dp][x] += sum[0][x], o[2 * dp + 1][x] += sum[1][x];
          } else {  // the middle terms take the rows 8-15, which no head has
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
              const uint32_t w[4] = {lo[u][0], mid[u][0], lo[u][2], mid[u][2]};
              mma_bf16(sum[0], w, vf[u][0], vf[u][1]);
              mma_bf16(sum[1], w, vf[u][2], vf[u][3]);
            }
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
              for (int x = 0; x < 2; ++x) sum[z][x] += sum[z][x + 2], sum[z][x + 2] = 0.f;
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
              mma_bf16(sum[0], hi[u], vf[u][0], vf[u][1]);
              mma_bf16(sum[1], hi[u], vf[u][2], vf[u][3]);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) o[2 * dp][x] += sum[0][x], o[2 * dp + 1][x] += sum[1][x];
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int x = 0; x < kHalves; ++x) {
        l[x] += __shfl_xor_sync(~0u, l[x], 1);
        l[x] += __shfl_xor_sync(~0u, l[x], 2);
        const int i = row + 8 * x;
        if (i >= rows) continue;
        if (covered) {
          if (kSkip && (lane & 3) == 0) p.cuts[b * p.h + h0 + i] = 0;
          const float inv = l[x] == 0.f ? 0.f : 1.f / l[x];
          const int64_t to = b * p.out.sn + (h0 + i) * p.out.sh + col;
#pragma unroll
          for (int c = 0; c < kD / 8; ++c) {
            if (p.out_is_f32)
              *reinterpret_cast<float2*>(static_cast<float*>(p.out.ptr) + to + c * 8) =
                  make_float2(o[c][2 * x] * inv, o[c][2 * x + 1] * inv);
            else
              *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out.ptr) + to + c * 8) =
                  pack_bf16x2(o[c][2 * x] * inv, o[c][2 * x + 1] * inv);
          }
          if ((lane & 3) == 0) write_lse(p, b, h0 + i, m[x], l[x]);
        } else {
          if ((lane & 3) == 0) ml[warp][which][i] = make_float2(m[x], l[x]);
#pragma unroll
          for (int c = 0; c < kD / 8; ++c)
            *reinterpret_cast<float2*>(part + i * C::kPitch + col + c * 8) = make_float2(o[c][2 * x], o[c][2 * x + 1]);
        }
      }
    }
    if (!covered && lane == 0) part_of[warp][which] = make_int2(k, unit);
    if (++unit == units) unit = 0, ++k;
  }

  // ---- units in several warps: merge their parts, in order ----------------------------
  __syncthreads();
  // Lane z: part z & 1 of warp z >> 1. A unit's parts follow one another; the first one leads.
  const int2 own = (&part_of[0][0])[lane & (2 * kWarps - 1)];
  const uint32_t valid = __ballot_sync(~0u, lane < 2 * kWarps && own.x >= 0);
  const uint32_t before = valid & ((1u << lane) - 1u);
  const int prev = before != 0 ? 31 - __clz(before) : 0;
  const int prev_x = __shfl_sync(~0u, own.x, prev), prev_y = __shfl_sync(~0u, own.y, prev);
  const bool follows = before != 0 && prev_x == own.x && prev_y == own.y;
  const uint32_t leads = __ballot_sync(~0u, ((valid >> lane) & 1u) && !follows);
  // A warp per (unit, row), lane c four columns; lane z works out the weight of part z.
  const int items = __popc(leads) * rows;
  for (int item = warp; item < items; item += kWarps) {
    const int nth = item / rows, row = item - nth * rows;
    uint32_t rest_of = leads;
    for (int i = 0; i < nth; ++i) rest_of &= rest_of - 1;
    const int x = __ffs(rest_of) - 1;
    rest_of &= rest_of - 1;
    const uint32_t these = valid & ~((1u << x) - 1u) & (rest_of != 0 ? (1u << (__ffs(rest_of) - 1)) - 1u : ~0u);
    const bool one = (these >> lane) & 1u;
    const float2 e = one ? ml[lane >> 1][lane & 1][row] : make_float2(-INFINITY, 0.f);
    float top = e.x;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    top = __shfl_sync(~0u, top, 0);
    const float f = one ? ex2_approx(e.x - (top == -INFINITY ? 0.f : top)) : 0.f;
    float sum = one ? f * e.y : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    sum = __shfl_sync(~0u, sum, 0);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const int c = min(lane * 4, kD - 4);
    for (uint32_t zs = these; zs != 0; zs &= zs - 1) {
      const int z = __ffs(zs) - 1;
      const float g = __shfl_sync(~0u, f, z);
      const float4 u = *reinterpret_cast<const float4*>(
          smem + (z % 2 ? (z / 2) * C::kWarpRing : C::kRing + (z / 2) * C::kPart) + (row * C::kPitch + c) * 4);
      o = make_float4(fmaf(g, u.x, o.x), fmaf(g, u.y, o.y), fmaf(g, u.z, o.z), fmaf(g, u.w, o.w));
    }
    const int k_of = __shfl_sync(~0u, own.x, x), unit_of = __shfl_sync(~0u, own.y, x);
    const int cnt = pre[k_of + 1] - pre[k_of], begin = pre[k_of] * units + unit_of * cnt, end = begin + cnt;
    const int64_t b = who[k_of];
    const int hh = unit_of * group + head0 + row;
    if (begin >= t0 && end <= t1) {
      if (lane * 4 < p.d) write_out4(p, b, hh, lane * 4, o, sum);
      if (lane == 0) write_lse(p, b, hh, top, sum);
      if (kSkip && lane == 0) p.cuts[b * p.h + hh] = 0;
      continue;
    }
    const int slot = blockIdx.x * 2 + (begin < t0 ? 0 : 1);
    if (lane * 4 < p.d)
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(ws + wl.o) + ((int64_t)slot * C::kRows + row) * kD + lane * 4) = o;
    if (lane == 0) reinterpret_cast<float2*>(ws + wl.ml)[slot * 16 + row] = make_float2(top, sum);
    if (begin >= t0 && (kSkip || row == 0) && lane == 0) {
      // the CTA whose run holds the unit's last tile, at cost v: runs up to the `over`-th are one longer
      const int v = begin_cost(k_of) + (unit_of + 1) * (cnt + kUnitCost) - 1;
      const int last = v < over * (share + 1) ? v / (share + 1) : over + (v - over * (share + 1)) / share;
      if (row == 0) reinterpret_cast<Split*>(ws)[blockIdx.x] = Split{(int)b, unit_of, last * a.planes + plane, 0};
      if constexpr (kSkip) p.cuts[b * p.h + hh] = cut_record(blockIdx.x, last - cta + 1, a.planes);
    }
  }
}

// Joins the parts of the unit that begins in CTA blockIdx.x's run and goes on after it, query head blockIdx.y of it. The
// parts are dealt to the block's warps, a lane has 4 columns; then the warps' results are merged in order. A chain of
// three memory latencies (which unit, its parts, the result) as long as a warp has at most kJoinBatch parts.
constexpr int kJoinWarps = 8;
constexpr int kJoinBatch = 4;

template <bool kF32, int kD, int kHd>
__global__ void __launch_bounds__(kJoinWarps * 32)
    paged_join_kernel(const __grid_constant__ PagedDecodeParams p, const __grid_constant__ Launch a) {
  using C = Cfg<kF32, kD, kHd>;
  __shared__ float4 part[kJoinWarps][32];
  __shared__ float2 part_ml[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y, cta = blockIdx.x;
  grid_launch_dependents();
  grid_dependency_wait();
  const uint8_t* ws = static_cast<const uint8_t*>(p.ws);
  const WsLayout wl = ws_layout(C::kRows, kD);
  const Split sp = reinterpret_cast<const Split*>(ws)[cta];
  if (sp.last < 0) return;
  const int group = p.h / p.hkv, head = a.head0 + cta % a.planes * C::kRows + row;
  if (head >= group) return;
  // part 0 is this CTA's entry 1, part i the entry 0 of its plane's i-th CTA from here
  const int parts = (sp.last - cta) / a.planes + 1;
  const bool mine = lane * 4 < p.d;
  float top = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float2 e, float4 y) {
    const float mn = fmaxf(top, e.x), ref = mn == -INFINITY ? 0.f : mn;
    const float f = ex2_approx(top - ref), g = ex2_approx(e.x - ref);
    top = mn;
    sum = fmaf(sum, f, e.y * g);
    o = make_float4(fmaf(o.x, f, y.x * g), fmaf(o.y, f, y.y * g), fmaf(o.z, f, y.z * g), fmaf(o.w, f, y.w * g));
  };
  for (int i0 = warp; i0 < parts; i0 += kJoinWarps * kJoinBatch) {
    float2 e[kJoinBatch];
    float4 y[kJoinBatch];
#pragma unroll
    for (int z = 0; z < kJoinBatch; ++z) {
      const int i = i0 + z * kJoinWarps, slot = i == 0 ? cta * 2 + 1 : (cta + i * a.planes) * 2;
      e[z] = make_float2(-INFINITY, 0.f);
      y[z] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < parts) {
        e[z] = reinterpret_cast<const float2*>(ws + wl.ml)[slot * 16 + row];
        if (mine) y[z] = *reinterpret_cast<const float4*>(ws + wl.o + (((int64_t)slot * C::kRows + row) * kD + lane * 4) * 4);
      }
    }
#pragma unroll
    for (int z = 0; z < kJoinBatch; ++z) add(e[z], y[z]);
  }
  if (warp > 0) {
    part[warp][lane] = o;
    if (lane == 0) part_ml[warp] = make_float2(top, sum);
  }
  __syncthreads();
  if (warp > 0) return;
  for (int w = 1; w < min(kJoinWarps, parts); ++w) add(part_ml[w], part[w][lane]);
  const int hh = sp.hk * group + head;
  if (lane == 0) write_lse(p, sp.b, hh, top, sum);
  if (p.cuts != nullptr && lane == 0) p.cuts[(int64_t)sp.b * p.h + hh] = 0;  // no longer
  if (mine) write_out4(p, sp.b, hh, lane * 4, o, sum);
}

// The most that one request's units can cost.
int64_t request_cost(int64_t keys, int64_t units, int tile) { return ((keys + tile - 1) / tile + 1 + kUnitCost) * units; }

template <bool kF32, int kD, int kHd, bool kSkip = false>
cudaError_t launch(const PagedDecodeParams& p, cudaStream_t s, int* nlaunch) {
  using C = Cfg<kF32, kD, kHd>;
  static PerContext<int> cache;
  int ctas = 0;
  cudaError_t e = cache.get(
      [](int* v) {
        cudaError_t r = cudaFuncSetAttribute(paged_decode_kernel<kF32, kD, kHd, kSkip>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             C::kSmem);
        if (r != cudaSuccess) return r;
        int sms = 0;
        if ((r = device_sm_count(&sms)) != cudaSuccess) return r;
        *v = sms < kMaxCtas ? sms : kMaxCtas;
        return r;
      },
      &ctas);
  if (e != cudaSuccess) return e;
  const int group = p.h / p.hkv;
  Launch a;
  a.sl2 = p.scale * kLog2e;
  const int64_t keys = (int64_t)p.max_pages * p.page;
  a.split = keys > kWholeTiles * C::kKeys;
  // Requests per launch: their tiles and unit costs have to stay countable in 31 bits.
  int64_t at_once = ((int64_t(1) << 31) - 1) / request_cost(keys, p.hkv, C::kKeys);
  if (at_once > kMaxRequests) at_once = kMaxRequests;
  // Of a launch, so that a plane keeps CTAs enough to cut its work among. 300 heads to a K/V head, 16 requests of 4k-8k
  // keys: 155 us; 8: 161, 4: 183, 32: 136 us.
  constexpr int kMaxPlanes = 16;
  // Of requests whose first keys are left out the caller joins what is cut, unless the rounds share the workspace.
  const bool join_here = !kSkip || group > kMaxPlanes * C::kRows || p.n > at_once;
  for (a.head0 = 0; a.head0 < group; a.head0 += kMaxPlanes * C::kRows) {
    const int left = (group - a.head0 + C::kRows - 1) / C::kRows;
    a.planes = left < kMaxPlanes ? left : kMaxPlanes;
    const unsigned grid = (unsigned)(ctas / a.planes * a.planes);
    for (int64_t r0 = 0; r0 < p.n; r0 += at_once) {
      a.r0 = (int)r0;
      a.n = (int)(p.n - r0 < at_once ? p.n - r0 : at_once);
      e = launch_dependent(paged_decode_kernel<kF32, kD, kHd, kSkip>, dim3(grid), kThreads, C::kSmem, s, p, a);
      if (e != cudaSuccess) return e;
      *nlaunch += 1;
      if (!a.split || !join_here) continue;
      const dim3 join(grid, (unsigned)(group < C::kRows ? group : C::kRows));
      if ((e = launch_dependent(paged_join_kernel<kF32, kD, kHd>, join, kJoinWarps * 32, 0, s, p, a)) != cudaSuccess)
        return e;
      *nlaunch += 1;
    }
  }
  return cudaSuccess;
}

}  // namespace

// The elements of a row in the kernels.
static int row_elements(int64_t d, bool is_f32) { return is_f32 && d <= 32 ? 32 : d <= 64 ? 64 : 128; }

size_t paged_decode_workspace(int64_t, int64_t, int64_t d, int64_t max_keys) {
  // Without the type: of the shorter of their uncut lengths.
  if (max_keys <= kWholeTiles * std::min(tile_keys(row_elements(d, true), true), tile_keys(row_elements(d, false), false)))
    return 0;
  return ws_layout(16, d <= 64 ? 64 : 128).total;
}

bool paged_decode_fits(int64_t hkv, int64_t d, bool is_f32, int64_t max_keys) {
  return request_cost(max_keys, hkv, tile_keys(row_elements(d, is_f32), is_f32)) < (int64_t(1) << 31);
}

// The smallest kernel that holds the group. bf16, 4 heads: 8 rows against 16, one request of 159 keys 5.7, 6.1 us, one of
// 8k keys 9.3, 9.8 us, large batches within 1%. f32: 1, 4, 8 rows for one head, 33 requests with a window 28.1, 31.5, 38.9
// us; 4, 8 rows for 4 heads, a large batch 237, 360 us. (The row's elements: d = 32 in 32, 64 a large batch 77.6, 94.6 us;
// d = 64 in 64, 128 121, 137 us.)
template <bool kF32, int kD>
static cudaError_t launch_heads(const PagedDecodeParams& p, cudaStream_t s, int* nlaunch) {
  const int group = p.h / p.hkv;
  if constexpr (!kF32) {
    return group <= 8 ? launch<false, kD, 8>(p, s, nlaunch) : launch<false, kD, 16>(p, s, nlaunch);
  } else {
    return group == 1   ? launch<true, kD, 1>(p, s, nlaunch)
           : group <= 4 ? launch<true, kD, 4>(p, s, nlaunch)
                        : launch<true, kD, 8>(p, s, nlaunch);
  }
}

template <int kD>
static cudaError_t launch_rest(const PagedDecodeParams& p, cudaStream_t s, int* nlaunch) {
  return p.h / p.hkv <= 8 ? launch<false, kD, 8, true>(p, s, nlaunch) : launch<false, kD, 16, true>(p, s, nlaunch);
}

cudaError_t launch_paged_decode_rest(const PagedDecodeParams& p, cudaStream_t s, int* nlaunch) {
  return p.d == 64 ? launch_rest<64>(p, s, nlaunch) : launch_rest<128>(p, s, nlaunch);
}

DecodeParts paged_decode_parts(int64_t h, int64_t hkv, int64_t d) {
  const int rows = h / hkv <= 8 ? 8 : 16;
  const WsLayout w = ws_layout(rows, row_elements(d, false));
  return DecodeParts{w.ml, w.o, rows};
}

cudaError_t launch_paged_decode(const PagedDecodeParams& p, cudaStream_t s, int* nlaunch) {
  if (!p.is_f32) return p.d == 64 ? launch_heads<false, 64>(p, s, nlaunch) : launch_heads<false, 128>(p, s, nlaunch);
  switch (row_elements(p.d, true)) {
    case 32: return launch_heads<true, 32>(p, s, nlaunch);
    case 64: return launch_heads<true, 64>(p, s, nlaunch);
    default: return launch_heads<true, 128>(p, s, nlaunch);
  }
}

}  // namespace bea
