// Attention of one new token per request over a paged K/V cache.
//
// out = sum_j p_j v_j / sum_j p_j with p_j = exp(scale q.k_j - m): one pass over
// the visible keys with a running maximum m and sum (online softmax), every key
// and value read once. HBM-bound: 2 d (K and V) elements a key and K/V head
// against 4 d g flops, g = h / h_kv query heads reading the same key.
//
// Work. A UNIT is one (request, K/V head, block of up to kRows of the group's
// query heads); its visible keys are cut into tiles of kKeys. The tiles of all
// units, request by request, make one list, and CTA c of G takes the c-th of G
// runs of it, each warp of the CTA an eighth of that, whatever the lengths are:
// nothing about them is known on the host. Every CTA finds its run from the
// lengths alone (a scan of tiles per request in shared memory). The runs cost
// the same: a unit counts as its tiles and kUnitCost more, for its queries and
// its output. A warp that covers a unit writes it; parts of a unit in several
// warps of a CTA are merged through shared memory when the warps are done, and
// parts in several CTAs go to the workspace as (O, m, l), which a second kernel
// joins in a fixed order (no atomics: the same call gives the same bits). If no
// unit is longer than kWholeTiles the CTAs' runs end at unit borders instead, and
// where the host sees that from the table's width it launches no second kernel.
//
// A warp streams its tiles by cp.async into a ring of its own, running ahead over
// unit borders, so no barrier stands before the end. Rows of a tile that no key
// of the request fills (behind its length, before its window, in a bad page)
// arrive as zeros and their scores are masked, so what those places hold in
// memory does not matter.
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
constexpr int kWholeTiles = 32;     // units up to this long are not cut
constexpr int kUnitCost = 2;        // of a unit, in tiles, besides its tiles
constexpr int kMinCost = 2 * kWarps;  // of a CTA's run, as long as there are fewer than G such runs
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <bool kF32, int kD>
struct Cfg {
  static constexpr int kKeys = kF32 ? 8 : 16;  // keys of a tile
  static constexpr int kRows = kF32 ? 8 : 16;  // query heads of a unit
  static constexpr int kEs = kF32 ? 4 : 2;
  static constexpr int kRowBytes = kD * kEs;
  static constexpr int kStageBytes = 2 * kKeys * kRowBytes;  // K then V
  static constexpr int kStages = 16384 / kStageBytes;       // 16 KB in flight or in use per warp
  static constexpr int kWarpRing = kStages * kStageBytes;
  static constexpr int kRing = kWarps * kWarpRing;
  static constexpr int kPitch = kD + 8;  // floats a row of a part: 8 rows x 4 lanes fall on different banks
  static constexpr int kPart = kRows * kPitch * 4;
  static constexpr int kHeads = kWarps * kPart;  // a warp's first part; its last one takes its ring's place
  static constexpr int kQ = kF32 ? kWarps * kRows * kD * 4 : 0;
  static constexpr int kP = kF32 ? kWarps * kKeys * kRows * 4 : 0;
  static constexpr int kSmem = kRing + kHeads + kQ + kP;
  // The 16-byte pieces of row r are stored at piece ^ swizzle(r): the eight rows an ldmatrix reads (bf16), the two
  // rows by four pieces a quarter-warp reads (f32) fall on different banks.
  __host__ __device__ static constexpr int swizzle(int r) { return kF32 ? ((r & 1) << 2) | ((r & 7) >> 1) : r & 7; }
  static_assert(kPart <= kWarpRing, "a part takes the place of its warp's ring");
};

// Workspace: [kMaxCtas] descriptors | [kMaxCtas][2][16] (m, l) | [kMaxCtas][2][rows][D] O. Entry 0 of a CTA is a
// unit that began before its run, entry 1 one that begins in the run and goes on after it.
struct Split {
  int b, unit, last, pad;  // last: the CTA that ends the unit; -1: nothing begins here that goes on
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
  int mtiles;    // blocks of query heads per K/V head
  int units;     // per request: h_kv * mtiles
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

// The first visible key of a request of `len` keys.
__device__ __forceinline__ int first_key(int len, int left) { return left >= len ? 0 : len - 1 - left; }

// The last index with key(index) <= x, key rising, key(0) <= x.
template <typename F>
__device__ __forceinline__ int last_below(int n, int64_t x, F key) {
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

template <bool kF32, int kD>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(const __grid_constant__ PagedDecodeParams p, const __grid_constant__ Launch a) {
  using C = Cfg<kF32, kD>;
  extern __shared__ __align__(128) uint8_t smem[];
  // requests with a visible key, in order: tiles of a unit summed over those before, number, length
  __shared__ int pre[kMaxRequests + 1], who[kMaxRequests], lens[kMaxRequests];
  __shared__ int warp_tiles[kWarps], warp_some[kWarps], warp_max[kWarps];
  __shared__ uint32_t masks[kWarps][C::kStages];
  __shared__ float2 ml[kWarps][2][16];  // of a warp's first and last part
  __shared__ int2 part_of[kWarps][2];   // (request, unit) of these parts, -1: none
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_launch_dependents();

  // ---- tiles per request, their sums, and this CTA's run [t0, t1) -----------------
  const int most = p.max_pages * p.page, units = a.units, grid = gridDim.x, cta = blockIdx.x;
  constexpr int kPer = kMaxRequests / kThreads;  // consecutive requests of a thread
  int len_of[kPer], tiles_of[kPer];
  int tiles_sum = 0, some = 0, longest = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = tid * kPer + i;
    len_of[i] = r < a.n ? p.lens[a.r0 + r] : 0;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    int len = len_of[i];
    if (len < 0 || len > most) {
      if (cta == 0) report_status(p.status, BEA_STATUS_PAGES);
      len = len_of[i] = len < 0 ? 0 : most;
    }
    tiles_of[i] = len > 0 ? (len + C::kKeys - 1) / C::kKeys - first_key(len, p.left) / C::kKeys : 0;
    tiles_sum += tiles_of[i];
    some += tiles_of[i] > 0;
    longest = max(longest, tiles_of[i]);
  }
  int tiles_inc = tiles_sum, some_inc = some;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(~0u, tiles_inc, o), y = __shfl_up_sync(~0u, some_inc, o);
    if (lane >= o) tiles_inc += x, some_inc += y;
  }
  longest = __reduce_max_sync(~0u, longest);
  if (lane == 31) warp_tiles[warp] = tiles_inc, warp_some[warp] = some_inc, warp_max[warp] = longest;
  if (lane < 2) part_of[warp][lane] = make_int2(-1, -1);
  __syncthreads();
  int run = 0, count = 0, at_tiles = tiles_inc - tiles_sum, at = some_inc - some;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) at_tiles += warp_tiles[w], at += warp_some[w];
    run += warp_tiles[w];
    count += warp_some[w];
    longest = max(longest, warp_max[w]);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (tiles_of[i] == 0) continue;
    pre[at] = at_tiles;
    who[at] = a.r0 + tid * kPer + i;
    lens[at++] = len_of[i];
    at_tiles += tiles_of[i];
  }
  if (tid == 0) pre[count] = run;
  // requests without a visible key
  if (count < a.n) {
    for (int r = cta; r < a.n; r += grid) {
      const int len = p.lens[a.r0 + r];
      if (len > 0 && most > 0) continue;
      const int64_t b = a.r0 + r;
      for (int i = tid; i < p.h * p.d; i += kThreads) {
        const int hh = i / p.d;
        const int64_t to = b * p.out.sn + hh * p.out.sh + (i - hh * p.d);
        if (p.out_is_f32)
          static_cast<float*>(p.out.ptr)[to] = 0.f;
        else
          static_cast<__nv_bfloat16*>(p.out.ptr)[to] = __float2bfloat16(0.f);
      }
      for (int i = tid; i < p.h; i += kThreads) p.lse.ptr[b * p.lse.sn + i * p.lse.sh] = -INFINITY;
    }
  }
  __syncthreads();

  // Costs. Unit u of the k-th request costs its tiles and kUnitCost before them.
  const int64_t cost = (int64_t)(run + kUnitCost * count) * units;
  const int ctas = (int)min((int64_t)grid, max((int64_t)1, cost / kMinCost));
  const bool whole = longest <= kWholeTiles;
  auto begin_cost = [&](int k) { return (int64_t)(pre[k] + kUnitCost * k) * units; };
  // where CTA c's run begins, as a cost
  auto border = [&](int c) {
    if (c >= ctas) return cost;
    int64_t v = cost * c / ctas;
    if (whole && v > 0) {
      const int k = last_below(count, v, begin_cost);
      const int each = pre[k + 1] - pre[k] + kUnitCost;
      const int64_t in = v - begin_cost(k);
      v += (in % each) * 2 < each ? -(in % each) : each - in % each;
    }
    return v;
  };
  // the first tile that is not before cost v
  auto tile_at = [&](int64_t v) {
    if (v >= cost) return run * units;
    const int k = last_below(count, v, begin_cost);
    const int cnt = pre[k + 1] - pre[k], in = (int)(v - begin_cost(k)), unit = in / (cnt + kUnitCost);
    return pre[k] * units + unit * cnt + max(0, in - unit * (cnt + kUnitCost) - kUnitCost);
  };
  const WsLayout wl = ws_layout(C::kRows, kD);
  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  if (a.split && tid == 0) reinterpret_cast<Split*>(ws)[cta] = Split{0, 0, -1, 0};
  if (cta >= ctas || count == 0) return;
  const int64_t v0 = border(cta), v1 = border(cta + 1);
  if (v0 >= v1) return;
  const int t0 = tile_at(v0), t1 = tile_at(v1);
  const int w0 = tile_at(v0 + (v1 - v0) * warp / kWarps), w1 = tile_at(v0 + (v1 - v0) * (warp + 1) / kWarps);

  // ---- loads: the i-th tile of this warp is tile w0 + i -------------------------------
  auto first_tile = [&](int k) { return (int64_t)pre[k] * units; };
  const uint32_t ring = smem_u32(smem) + warp * C::kWarpRing;
  const int group = p.h / p.hkv;
  const int mine = w1 - w0;
  const bool one_page = p.page % C::kKeys == 0;  // a tile lies in one page
  // Descriptors of this warp's next 32 tiles, one per lane.
  int d_b = 0, d_hk = 0, d_key = 0;
  int64_t d_k = 0, d_v = 0;
  uint32_t d_mask = 0;
  auto describe = [&](int i) {
    d_mask = 0;
    d_k = d_v = 0;
    if (i >= mine) return;
    const int t = w0 + i;
    const int k = last_below(count, t, first_tile);
    const int cnt = pre[k + 1] - pre[k], in = t - pre[k] * units, unit = in / cnt;
    const int len = lens[k], first = first_key(len, p.left);
    d_b = who[k];
    d_hk = unit / a.mtiles;
    d_key = (first / C::kKeys + (in - unit * cnt)) * C::kKeys;
    // rows of the tile that are visible
    const int lo = max(first - d_key, 0), hi = min(len - d_key, C::kKeys);
    d_mask = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
    if (one_page) {
      const int pg = d_key / p.page, off = d_key - pg * p.page;
      const int id = p.table[d_b * p.table_stride + pg];
      if (id < 0 || id >= p.num_pages) {
        report_status(p.status, BEA_STATUS_PAGES);
        d_mask = 0;
      } else {
        d_k = id * p.kc.sn + off * p.kc.sl + d_hk * p.kc.sh;
        d_v = id * p.vc.sn + off * p.vc.sl + d_hk * p.vc.sh;
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
      const int pg = key / p.page;
      n_off = key - pg * p.page;
      n_id = max(p.table[b * p.table_stride + pg], -1);
    }
  };
  auto load = [&](int i) {
    if (i < mine) {
      const int j = i & 31, stage = i % C::kStages;
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
          k_row = n_id * p.kc.sn + n_off * p.kc.sl + hk * p.kc.sh;
          v_row = n_id * p.vc.sn + n_off * p.vc.sl + hk * p.vc.sh;
        } else if (n_id != INT32_MIN) {
          report_status(p.status, BEA_STATUS_PAGES);
        }
        mask = __ballot_sync(~0u, ok);
      }
      if (lane == 0) masks[warp][stage] = mask;
      constexpr int kChunks = kD * C::kEs / 16;                 // 16-byte pieces of a row
      constexpr int kStep = 32 / kChunks;                       // rows per instruction
      const int chunk = lane % kChunks, sub = lane / kChunks;
      const bool in_row = !kF32 || chunk * 4 < p.d;
#pragma unroll
      for (int it = 0; it < C::kKeys / kStep; ++it) {
        const int row = it * kStep + sub;
        const bool read = (mask >> row) & 1u;
        int64_t ka = k_at + row * p.kc.sl, va = v_at + row * p.vc.sl;
        if (!one_page) ka = __shfl_sync(~0u, k_row, row), va = __shfl_sync(~0u, v_row, row);
        const uint32_t to = row * C::kRowBytes + ((chunk ^ C::swizzle(row)) << 4);
        const char* ks = static_cast<const char*>(p.kc.ptr) + ka * C::kEs + chunk * 16;
        const char* vs = static_cast<const char*>(p.vc.ptr) + va * C::kEs + chunk * 16;
        if (in_row) {
          cp_async16(kd + to, read ? ks : p.q.ptr, read);
          cp_async16(vd + to, read ? vs : p.q.ptr, read);
        }
      }
      if (!one_page) look_up(i + 1);
    }
    cp_async_commit();  // an empty group where there is no tile, so that groups count tiles
  };
  if (!one_page) look_up(0);
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) load(i);

  // ---- unit by unit ----------------------------------------------------------------
  float* head = reinterpret_cast<float*>(smem + C::kRing + warp * C::kPart);
  float* tail = reinterpret_cast<float*>(smem + warp * C::kWarpRing);
  float* q_smem = reinterpret_cast<float*>(smem + C::kRing + C::kHeads) + warp * C::kRows * kD;
  float* p_smem = reinterpret_cast<float*>(smem + C::kRing + C::kHeads + C::kQ) + warp * C::kKeys * C::kRows;
  int done = 0;
  int k = last_below(count, w0, first_tile);
  int unit = (w0 - pre[k] * units) / (pre[k + 1] - pre[k]);
  while (done < mine) {
    const int cnt = pre[k + 1] - pre[k], begin = pre[k] * units + unit * cnt, end = begin + cnt;
    const int todo = min(end, w1) - w0;  // this warp's tiles up to the unit's end
    const int64_t b = who[k];
    const int hk = unit / a.mtiles, mi = unit - hk * a.mtiles;
    const int h0 = hk * group + mi * C::kRows, rows = min(C::kRows, group - mi * C::kRows);
    const bool covered = begin >= w0 && end <= w1;
    const int which = begin < w0 ? 0 : 1;
    float* part = which == 0 ? head : tail;

    if constexpr (kF32) {
      // Scores: lane (key, quarter) takes every fourth 16-byte piece of its key's row. Output: lane owns 4 columns.
      float m[C::kRows], l[C::kRows];  // l: this lane's keys only, quarter 0 counts
      float4 o[C::kRows];
#pragma unroll
      for (int i = 0; i < C::kRows; ++i) m[i] = -INFINITY, l[i] = 0.f, o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      const float* q = static_cast<const float*>(p.q.ptr) + b * p.q.sn + h0 * p.q.sh;
      __syncwarp();
      for (int i = 0; i < rows; ++i)
        if (lane * 4 < p.d)
          *reinterpret_cast<float4*>(q_smem + i * kD + lane * 4) =
              *reinterpret_cast<const float4*>(q + i * p.q.sh + lane * 4);
      __syncwarp();
      const int key = lane >> 2, quarter = lane & 3, sw = C::swizzle(key), pieces = p.d >> 2;
      const bool column = lane * 4 < kD;
      for (; done < todo; ++done) {
        const int stage = done % C::kStages;
        load(done + C::kStages - 1);
        cp_async_wait<C::kStages - 1>();
        __syncwarp();
        const uint8_t* kt = smem + warp * C::kWarpRing + stage * C::kStageBytes;
        const uint8_t* vt = kt + C::kKeys * C::kRowBytes;
        const bool see = (masks[warp][stage] >> key) & 1u;
        float s[C::kRows];
#pragma unroll
        for (int i = 0; i < C::kRows; ++i) s[i] = 0.f;
        for (int c = quarter; c < pieces; c += 4) {
          const float4 x = *reinterpret_cast<const float4*>(kt + key * C::kRowBytes + ((c ^ sw) << 4));
#pragma unroll
          for (int i = 0; i < C::kRows; ++i) {
            if (i < rows) {
              const float4 y = *reinterpret_cast<const float4*>(q_smem + i * kD + c * 4);
              s[i] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s[i]))));
            }
          }
        }
#pragma unroll
        for (int i = 0; i < C::kRows; ++i) {
          if (i < rows) {
            s[i] += __shfl_xor_sync(~0u, s[i], 1);
            s[i] += __shfl_xor_sync(~0u, s[i], 2);
            s[i] = see ? s[i] * a.sl2 : -INFINITY;
            float top = s[i];
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
            if (top > m[i]) {
              const float w = ex2_approx(m[i] - top);
              m[i] = top;
              l[i] *= w;
              o[i] = make_float4(o[i].x * w, o[i].y * w, o[i].z * w, o[i].w * w);
            }
            const float e = ex2_approx(s[i] - (m[i] == -INFINITY ? 0.f : m[i]));
            if (quarter == 0) {
              l[i] += e;
              p_smem[key * C::kRows + i] = e;
            }
          }
        }
        __syncwarp();
        if (column) {
#pragma unroll
          for (int j = 0; j < C::kKeys; ++j) {
            const float4 v = *reinterpret_cast<const float4*>(vt + j * C::kRowBytes + ((lane ^ C::swizzle(j)) << 4));
#pragma unroll
            for (int i = 0; i < C::kRows; ++i) {
              if (i < rows) {
                const float e = p_smem[j * C::kRows + i];
                o[i] = make_float4(fmaf(e, v.x, o[i].x), fmaf(e, v.y, o[i].y), fmaf(e, v.z, o[i].z), fmaf(e, v.w, o[i].w));
              }
            }
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < C::kRows; ++i) {
        if (i < rows) {
          l[i] += __shfl_xor_sync(~0u, l[i], 4);
          l[i] += __shfl_xor_sync(~0u, l[i], 8);
          l[i] += __shfl_xor_sync(~0u, l[i], 16);
          l[i] = __shfl_sync(~0u, l[i], 0);
          if (covered) {
            const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
            if (lane * 4 < p.d)
              *reinterpret_cast<float4*>(static_cast<float*>(p.out.ptr) + b * p.out.sn + (h0 + i) * p.out.sh + lane * 4) =
                  make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv);
            if (lane == 0)
              p.lse.ptr[b * p.lse.sn + (h0 + i) * p.lse.sh] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
          } else {
            if (lane == 0) ml[warp][which][i] = make_float2(m[i], l[i]);
            if (lane * 4 < p.d) *reinterpret_cast<float4*>(part + i * C::kPitch + lane * 4) = o[i];
          }
        }
      }
    } else {
      // m16n8k16: rows are query heads, S = Q K^T leaves P in the layout the second product takes as its A operand.
      float o[kD / 8][4];
#pragma unroll
      for (int i = 0; i < kD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      const int row = lane >> 2, col = (lane & 3) * 2;
      uint32_t qf[kD / 16][4];
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q.ptr) + b * p.q.sn + h0 * p.q.sh;
#pragma unroll
      for (int ks = 0; ks < kD / 16; ++ks)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int i = row + (x & 1) * 8, c = ks * 16 + (x >> 1) * 8 + col;
          qf[ks][x] = i < rows ? *reinterpret_cast<const uint32_t*>(q + i * p.q.sh + c) : 0u;
        }
      for (; done < todo; ++done) {
        const int stage = done % C::kStages;
        load(done + C::kStages - 1);
        cp_async_wait<C::kStages - 1>();
        __syncwarp();
        const uint32_t kt = ring + stage * C::kStageBytes, vt = kt + C::kKeys * C::kRowBytes;
        const uint32_t mask = masks[warp][stage];
        float s[2][4] = {};
#pragma unroll
        for (int ks = 0; ks < kD / 16; ++ks) {
          uint32_t kf[4];
          const int kr = (lane & 7) + ((lane >> 4) << 3), chunk = 2 * ks + ((lane >> 3) & 1);
          ldsm4(kt + kr * C::kRowBytes + ((chunk ^ C::swizzle(kr)) << 4), kf);
          mma_bf16(s[0], qf[ks], kf[0], kf[1]);
          mma_bf16(s[1], qf[ks], kf[2], kf[3]);
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const bool see = (mask >> (nb * 8 + col + (x & 1))) & 1u;
            s[nb][x] = see ? s[nb][x] * a.sl2 : -INFINITY;
            top[x >> 1] = fmaxf(top[x >> 1], s[nb][x]);
          }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 1));
          top[x] = fmaxf(top[x], __shfl_xor_sync(~0u, top[x], 2));
        }
        // O and l are rescaled only when a maximum grows by more than 2^8: the reference value then in use
        // cancels in the end, and P stays below 2^8.
        if (__any_sync(~0u, top[0] > m[0] + 8.f || top[1] > m[1] + 8.f)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float mn = fmaxf(m[x], top[x]);
            const float w = mn == -INFINITY ? 1.f : ex2_approx(m[x] - mn);
            m[x] = mn;
            l[x] *= w;
#pragma unroll
            for (int i = 0; i < kD / 8; ++i) o[i][2 * x] *= w, o[i][2 * x + 1] *= w;
          }
        }
        // P as two bf16 terms: the first 8 bits truncated, the rest rounded (2^-15 of P left over, where one term
        // would leave 2^-8). The second term is kept above 0, so that an infinite value stays infinite.
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float ref = m[x] == -INFINITY ? 0.f : m[x];
            const float p0 = ex2_approx(s[nb][2 * x] - ref), p1 = ex2_approx(s[nb][2 * x + 1] - ref);
            l[x] += p0 + p1;
            const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
            hi[nb * 2 + x] = __byte_perm(u0, u1, 0x7632);
            const float r0 = fmaxf(p0 - __uint_as_float(u0 & 0xFFFF0000u), p0 * 0x1p-20f);
            const float r1 = fmaxf(p1 - __uint_as_float(u1 & 0xFFFF0000u), p1 * 0x1p-20f);
            lo[nb * 2 + x] = pack_bf16x2(r0, r1);
          }
#pragma unroll
        for (int dp = 0; dp < kD / 16; ++dp) {
          uint32_t vf[4];
          const int vr = (lane & 7) + (((lane >> 3) & 1) << 3), chunk = 2 * dp + (lane >> 4);
          ldsm4_t(vt + vr * C::kRowBytes + ((chunk ^ C::swizzle(vr)) << 4), vf);
          mma_bf16(o[2 * dp], hi, vf[0], vf[1]);
          mma_bf16(o[2 * dp + 1], hi, vf[2], vf[3]);
          mma_bf16(o[2 * dp], lo, vf[0], vf[1]);
          mma_bf16(o[2 * dp + 1], lo, vf[2], vf[3]);
        }
        __syncwarp();
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(~0u, l[x], 1);
        l[x] += __shfl_xor_sync(~0u, l[x], 2);
        const int i = row + 8 * x;
        if (i >= rows) continue;
        if (covered) {
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
          if ((lane & 3) == 0)
            p.lse.ptr[b * p.lse.sn + (h0 + i) * p.lse.sh] = l[x] == 0.f ? -INFINITY : (m[x] + log2f(l[x])) * kLn2;
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
  const int quads = p.d >> 2;
  const int2* parts = &part_of[0][0];
  for (int x = 0; x < 2 * kWarps;) {
    const int2 of = parts[x];
    if (of.x < 0) {
      ++x;
      continue;
    }
    int y = x + 1;  // parts [x, y) are this unit's
    while (y < 2 * kWarps && (parts[y].x < 0 || (parts[y].x == of.x && parts[y].y == of.y))) ++y;
    const int cnt = pre[of.x + 1] - pre[of.x], begin = pre[of.x] * units + of.y * cnt, end = begin + cnt;
    const int64_t b = who[of.x];
    const int hk = of.y / a.mtiles, mi = of.y - hk * a.mtiles;
    const int h0 = hk * group + mi * C::kRows, rows = min(C::kRows, group - mi * C::kRows);
    const bool complete = begin >= t0 && end <= t1;
    const int slot = cta * 2 + (begin < t0 ? 0 : 1);
    for (int i = tid; i < rows * quads; i += kThreads) {
      const int row = i / quads, c = (i - row * quads) * 4;
      float top = -INFINITY;
      for (int z = x; z < y; ++z)
        if (parts[z].x >= 0) top = fmaxf(top, ml[z >> 1][z & 1][row].x);
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int z = x; z < y; ++z) {
        if (parts[z].x < 0) continue;
        const float2 e = ml[z >> 1][z & 1][row];
        const float f = ex2_approx(e.x - ref);
        const float* from = reinterpret_cast<const float*>(smem + ((z & 1) ? (z >> 1) * C::kWarpRing : C::kRing + (z >> 1) * C::kPart));
        const float4 u = *reinterpret_cast<const float4*>(from + row * C::kPitch + c);
        sum = fmaf(f, e.y, sum);
        o = make_float4(fmaf(f, u.x, o.x), fmaf(f, u.y, o.y), fmaf(f, u.z, o.z), fmaf(f, u.w, o.w));
      }
      if (complete) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t to = b * p.out.sn + (h0 + row) * p.out.sh + c;
        if (p.out_is_f32) {
          *reinterpret_cast<float4*>(static_cast<float*>(p.out.ptr) + to) =
              make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        } else {
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out.ptr) + to) =
              make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        }
        if (c == 0)
          p.lse.ptr[b * p.lse.sn + (h0 + row) * p.lse.sh] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(ws + wl.o) + ((int64_t)slot * C::kRows + row) * kD + c) = o;
        if (c == 0) reinterpret_cast<float2*>(ws + wl.ml)[slot * 16 + row] = make_float2(top, sum);
      }
    }
    if (!complete && begin >= t0 && tid == 0) {
      // the CTA whose run holds the unit's last tile, at cost v: the last one that begins there or before
      const int64_t v = begin_cost(of.x) + (int64_t)(of.y + 1) * (cnt + kUnitCost) - 1;
      int last = (int)(v * ctas / cost);
      while (last + 1 < ctas && cost * (last + 1) / ctas <= v) ++last;
      while (cost * last / ctas > v) --last;
      reinterpret_cast<Split*>(ws)[cta] = Split{(int)b, of.y, last, 0};
    }
    x = y;
  }
}

// Joins the parts of unit that begins in CTA blockIdx.x's run, query head blockIdx.y of it: the parts are dealt to the
// block's warps, each lane 4 columns, then the warps' results are summed in order.
constexpr int kJoinWarps = 8;

template <bool kF32, int kD>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const __grid_constant__ PagedDecodeParams p,
                                                                      const __grid_constant__ Launch a) {
  using C = Cfg<kF32, kD>;
  __shared__ float4 part[kJoinWarps][32];
  __shared__ float sums[kJoinWarps], tops[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y, cta = blockIdx.x;
  grid_dependency_wait();
  const uint8_t* ws = static_cast<const uint8_t*>(p.ws);
  const WsLayout wl = ws_layout(C::kRows, kD);
  const Split sp = reinterpret_cast<const Split*>(ws)[cta];
  if (sp.last < 0) return;
  const int group = p.h / p.hkv, hk = sp.unit / a.mtiles, mi = sp.unit - hk * a.mtiles;
  if (row >= min(C::kRows, group - mi * C::kRows)) return;
  const float2* ml = reinterpret_cast<const float2*>(ws + wl.ml);
  const float* os = reinterpret_cast<const float*>(ws + wl.o);
  // part 0 is this CTA's entry 1, part i the entry 0 of CTA + i
  const int parts = sp.last - cta + 1;
  auto slot = [&](int i) { return i == 0 ? cta * 2 + 1 : (cta + i) * 2; };
  float top = -INFINITY;
  for (int i = threadIdx.x; i < parts; i += kJoinWarps * 32) top = fmaxf(top, ml[slot(i) * 16 + row].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, tops[w]);
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool mine = lane * 4 < p.d;
#pragma unroll 8
  for (int i = warp; i < parts; i += kJoinWarps) {
    const float2 x = ml[slot(i) * 16 + row];
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mine) y = *reinterpret_cast<const float4*>(os + ((int64_t)slot(i) * C::kRows + row) * kD + lane * 4);
    const float f = ex2_approx(x.x - ref);
    sum = fmaf(f, x.y, sum);
    o = make_float4(fmaf(f, y.x, o.x), fmaf(f, y.y, o.y), fmaf(f, y.z, o.z), fmaf(f, y.w, o.w));
  }
  part[warp][lane] = o;
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  if (warp != 0) return;
  sum = sums[0];
  o = part[0][lane];
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) {
    const float4 y = part[w][lane];
    sum += sums[w];
    o = make_float4(o.x + y.x, o.y + y.y, o.z + y.z, o.w + y.w);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t b = sp.b;
  const int hh = hk * group + mi * C::kRows + row;
  if (lane == 0) p.lse.ptr[b * p.lse.sn + hh * p.lse.sh] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  if (!mine) return;
  const int64_t at = b * p.out.sn + hh * p.out.sh + lane * 4;
  if (p.out_is_f32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out.ptr) + at) =
        make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  } else {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out.ptr) + at) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  }
}

// The most that one request's units can cost.
int64_t request_cost(int64_t keys, int64_t units, int tile) { return ((keys + tile - 1) / tile + 1 + kUnitCost) * units; }

template <bool kF32, int kD>
cudaError_t launch(const PagedDecodeParams& p, cudaStream_t s, int* nlaunch) {
  using C = Cfg<kF32, kD>;
  static PerContext<int> cache;
  int ctas = 0;
  cudaError_t e = cache.get(
      [](int* v) {
        cudaError_t r = cudaFuncSetAttribute(paged_decode_kernel<kF32, kD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  a.mtiles = (group + C::kRows - 1) / C::kRows;
  a.units = p.hkv * a.mtiles;
  a.sl2 = p.scale * kLog2e;
  const int64_t keys = (int64_t)p.max_pages * p.page;
  a.split = keys > kWholeTiles * C::kKeys;
  // Requests per launch: their tiles and unit costs have to stay countable in 31 bits.
  int64_t at_once = ((int64_t(1) << 31) - 1) / request_cost(keys, a.units, C::kKeys);
  if (at_once > kMaxRequests) at_once = kMaxRequests;
  for (int64_t r0 = 0; r0 < p.n; r0 += at_once) {
    a.r0 = (int)r0;
    a.n = (int)(p.n - r0 < at_once ? p.n - r0 : at_once);
    paged_decode_kernel<kF32, kD><<<ctas, kThreads, C::kSmem, s>>>(p, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    *nlaunch += 1;
    if (!a.split) continue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)(group < C::kRows ? group : C::kRows));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, paged_join_kernel<kF32, kD>, p, a)) != cudaSuccess) return e;
    *nlaunch += 1;
  }
  return cudaSuccess;
}

}  // namespace

size_t paged_decode_workspace(int64_t, int64_t, int64_t d, int64_t max_keys) {
  // Without the type: the larger of the two kernels' needs, for the shorter of their uncut lengths.
  if (max_keys <= kWholeTiles * Cfg<true, 128>::kKeys) return 0;
  return ws_layout(16, d <= 64 ? 64 : 128).total;
}

bool paged_decode_fits(int64_t h, int64_t hkv, bool is_f32, int64_t max_keys) {
  const int rows = is_f32 ? Cfg<true, 128>::kRows : Cfg<false, 128>::kRows;
  const int64_t units = hkv * ((h / hkv + rows - 1) / rows);
  return request_cost(max_keys, units, is_f32 ? Cfg<true, 128>::kKeys : Cfg<false, 128>::kKeys) < (int64_t(1) << 31);
}

cudaError_t launch_paged_decode(const PagedDecodeParams& p, cudaStream_t s, int* nlaunch) {
  if (p.is_f32) return p.d <= 64 ? launch<true, 64>(p, s, nlaunch) : launch<true, 128>(p, s, nlaunch);
  return p.d == 64 ? launch<false, 64>(p, s, nlaunch) : launch<false, 128>(p, s, nlaunch);
}

}  // namespace bea
