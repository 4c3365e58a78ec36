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
// equal runs of it, whatever the lengths are: nothing about them is known on the
// host. Every CTA finds its run from the lengths alone (a scan of tiles per
// request in shared memory). A unit that one CTA covers is written by it; of a
// unit that is cut, each CTA leaves (O, m, l) in the workspace and a second
// kernel joins them in a fixed order (no atomics: the same call gives the same
// bits). If no unit is longer than kWholeTiles the runs' ends are moved to
// unit borders instead, and if the host can see that from the table's width
// the second kernel is not launched.
//
// Inside a CTA each of the four warps takes every fourth tile of the run and
// streams it by cp.async into a ring of its own, running ahead over unit borders,
// so no barrier stands in the loop; at the end of a unit the warps' (O, m, l) are
// merged through shared memory. Rows of a tile that no key of the request fills
// (behind its length, before its window, in a bad page) arrive as zeros and their
// scores are masked, so what those places hold in memory does not matter.
#include <cuda_bf16.h>

#include "launch_cache.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace bea {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCtas = 304;       // two per SM
constexpr int kMaxRequests = 1024;  // per launch: their tile counts are scanned in shared memory
constexpr int kWholeTiles = 32;     // units up to this long are not cut
constexpr int kMinTiles = 2 * kWarps;  // of a CTA's run, as long as there are fewer than G such runs
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <bool kF32, int kD>
struct Cfg {
  static constexpr int kKeys = kF32 ? 8 : 16;  // keys of a tile
  static constexpr int kRows = kF32 ? 8 : 16;  // query heads of a unit
  static constexpr int kEs = kF32 ? 4 : 2;
  static constexpr int kRowBytes = kD * kEs;
  static constexpr int kStages = kF32 ? 2 : (kD == 64 ? 4 : 2);
  static constexpr int kStageBytes = 2 * kKeys * kRowBytes;  // K then V
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kPitch = kD + 8;  // floats a row of the merge buffer: 8 rows x 4 lanes fall on different banks
  static constexpr int kMerge = kWarps * kRows * kPitch * 4;
  static constexpr int kQ = kF32 ? kWarps * kRows * kD * 4 : 0;
  static constexpr int kP = kF32 ? kWarps * kKeys * kRows * 4 : 0;
  static constexpr int kSmem = kRing + kMerge + kQ + kP;
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

// The request of tile t: pre[b] * units <= t < pre[b + 1] * units.
__device__ __forceinline__ int request_of(const int* pre, int n, int units, int t) {
  const int x = t / units;
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid + 1] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

template <bool kF32, int kD>
__global__ void __launch_bounds__(kThreads, 2)
    paged_decode_kernel(const __grid_constant__ PagedDecodeParams p, const __grid_constant__ Launch a) {
  using C = Cfg<kF32, kD>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int pre[kMaxRequests + 1];  // tiles of a unit, summed over the requests before
  __shared__ int lens[kMaxRequests];
  __shared__ int warp_sum[kWarps], warp_max[kWarps];
  __shared__ uint32_t masks[kWarps][C::kStages];
  __shared__ float2 ml[kWarps][16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_launch_dependents();

  // ---- tiles per request, their sums, and this CTA's run [t0, t1) -----------------
  const int most = p.max_pages * p.page;
  int run = 0, longest = 0;
  for (int base = 0; base < a.n; base += kThreads) {
    const int r = base + tid;
    int tiles = 0;
    if (r < a.n) {
      int len = p.lens[a.r0 + r];
      if (len < 0 || len > most) {
        if (blockIdx.x == 0) report_status(p.status, BEA_STATUS_PAGES);
        len = len < 0 ? 0 : most;
      }
      lens[r] = len;
      if (len > 0) tiles = (len + C::kKeys - 1) / C::kKeys - first_key(len, p.left) / C::kKeys;
      longest = max(longest, tiles);
    }
    int inc = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int before = run;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += warp_sum[w];
      run += warp_sum[w];
    }
    if (r < a.n) pre[r + 1] = before + inc;
    __syncthreads();
  }
  if (tid == 0) pre[0] = 0;
  longest = __reduce_max_sync(~0u, longest);
  if (lane == 0) warp_max[warp] = longest;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) longest = max(longest, warp_max[w]);

  const int units = a.units, total = run * units, grid = gridDim.x, cta = blockIdx.x;
  const int ctas = min(grid, max(1, total / kMinTiles));
  const bool whole = longest <= kWholeTiles;
  auto border = [&](int c) {
    if (c >= ctas) return total;
    int t = (int)((int64_t)total * c / ctas);
    if (whole && t > 0) {
      const int b = request_of(pre, a.n, units, t);
      const int cnt = pre[b + 1] - pre[b], begin = pre[b] * units;
      t = begin + (t - begin) / cnt * cnt;
    }
    return t;
  };
  const int t0 = border(min(cta, ctas)), t1 = border(min(cta + 1, ctas));

  // requests without a visible key
  for (int r = cta; r < a.n; r += grid) {
    if (pre[r + 1] != pre[r]) continue;
    const int64_t b = a.r0 + r;
    for (int i = tid; i < p.h * p.d; i += kThreads) {
      const int hh = i / p.d;
      const int64_t at = b * p.out.sn + hh * p.out.sh + (i - hh * p.d);
      if (p.out_is_f32)
        static_cast<float*>(p.out.ptr)[at] = 0.f;
      else
        static_cast<__nv_bfloat16*>(p.out.ptr)[at] = __float2bfloat16(0.f);
    }
    for (int i = tid; i < p.h; i += kThreads) p.lse.ptr[b * p.lse.sn + i * p.lse.sh] = -INFINITY;
  }
  const WsLayout wl = ws_layout(C::kRows, kD);
  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  if (a.split && tid == 0) reinterpret_cast<Split*>(ws)[cta] = Split{0, 0, -1, 0};
  if (t0 >= t1) return;

  // ---- loads: the i-th tile of this warp is tile t0 + warp + 4 i ---------------------
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
  const int group = p.h / p.hkv;
  const int mine = (t1 - t0 - warp + kWarps - 1) / kWarps;  // may be <= 0
  const bool paged16 = p.page % C::kKeys == 0;              // a tile lies in one page
  // Descriptors of this warp's next 32 tiles, one per lane.
  int d_b = 0, d_hk = 0, d_key = 0;
  int64_t d_k = 0, d_v = 0;
  uint32_t d_mask = 0;
  auto describe = [&](int i) {
    d_mask = 0;
    d_k = d_v = 0;
    if (i >= mine) return;
    const int t = t0 + warp + kWarps * i;
    const int r = request_of(pre, a.n, units, t);
    const int cnt = pre[r + 1] - pre[r], in = t - pre[r] * units, unit = in / cnt;
    const int len = lens[r], first = first_key(len, p.left);
    d_b = a.r0 + r;
    d_hk = unit / a.mtiles;
    d_key = (first / C::kKeys + (in - unit * cnt)) * C::kKeys;
    // rows of the tile that are visible
    const int lo = max(first - d_key, 0), hi = min(len - d_key, C::kKeys);
    d_mask = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
    if (paged16) {
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
  auto load = [&](int i) {
    if (i < mine) {
      const int j = i & 31;
      if (j == 0) describe(i + lane);
      const int stage = i % C::kStages;
      const uint32_t kd = ring + stage * C::kStageBytes, vd = kd + C::kKeys * C::kRowBytes;
      uint32_t mask = __shfl_sync(~0u, d_mask, j);
      int64_t k_at = __shfl_sync(~0u, d_k, j), v_at = __shfl_sync(~0u, d_v, j);
      int64_t k_row = 0, v_row = 0;
      if (!paged16) {  // each row's own place
        const int b = __shfl_sync(~0u, d_b, j), hk = __shfl_sync(~0u, d_hk, j), key = __shfl_sync(~0u, d_key, j) + lane;
        bool ok = lane < C::kKeys && ((mask >> (lane & 15)) & 1u);
        if (ok) {
          const int pg = key / p.page, off = key - pg * p.page;
          const int id = p.table[b * p.table_stride + pg];
          ok = id >= 0 && id < p.num_pages;
          if (ok) {
            k_row = id * p.kc.sn + off * p.kc.sl + hk * p.kc.sh;
            v_row = id * p.vc.sn + off * p.vc.sl + hk * p.vc.sh;
          } else {
            report_status(p.status, BEA_STATUS_PAGES);
          }
        }
        mask = __ballot_sync(~0u, ok);
      }
      if (lane == 0) masks[warp][stage] = mask;
      if constexpr (kF32) {
#pragma unroll
        for (int row = 0; row < C::kKeys; ++row) {
          const bool read = (mask >> row) & 1u;
          int64_t ka = k_at + row * p.kc.sl, va = v_at + row * p.vc.sl;
          if (!paged16) ka = __shfl_sync(~0u, k_row, row), va = __shfl_sync(~0u, v_row, row);
          if (lane * 4 < p.d) {
            const uint32_t at = row * C::kRowBytes + ((lane ^ (((row & 1) << 2) | (row >> 1))) << 4);
            cp_async16(kd + at, read ? static_cast<const float*>(p.kc.ptr) + ka + lane * 4 : p.q.ptr, read);
            cp_async16(vd + at, read ? static_cast<const float*>(p.vc.ptr) + va + lane * 4 : p.q.ptr, read);
          }
        }
      } else {
        constexpr int kChunks = kD / 8, kStep = 32 / kChunks;  // rows per instruction
        const int chunk = lane % kChunks, sub = lane / kChunks;
#pragma unroll
        for (int it = 0; it < C::kKeys / kStep; ++it) {
          const int row = it * kStep + sub;
          const bool read = (mask >> row) & 1u;
          int64_t ka = k_at + row * p.kc.sl, va = v_at + row * p.vc.sl;
          if (!paged16) ka = __shfl_sync(~0u, k_row, row), va = __shfl_sync(~0u, v_row, row);
          const uint32_t at = row * C::kRowBytes + ((chunk ^ (row & 7)) << 4);
          cp_async16(kd + at, read ? static_cast<const __nv_bfloat16*>(p.kc.ptr) + ka + chunk * 8 : p.q.ptr, read);
          cp_async16(vd + at, read ? static_cast<const __nv_bfloat16*>(p.vc.ptr) + va + chunk * 8 : p.q.ptr, read);
        }
      }
    }
    cp_async_commit();  // an empty group where there is no tile, so that groups count tiles
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) load(i);

  // ---- unit by unit ----------------------------------------------------------------
  float* merge = reinterpret_cast<float*>(smem + C::kRing);
  float* q_smem = reinterpret_cast<float*>(smem + C::kRing + C::kMerge) + warp * C::kRows * kD;
  float* p_smem = reinterpret_cast<float*>(smem + C::kRing + C::kMerge + C::kQ) + warp * C::kKeys * C::kRows;
  int done = 0;  // tiles of this warp
  int r = request_of(pre, a.n, units, t0);
  int unit = (t0 - pre[r] * units) / (pre[r + 1] - pre[r]);
  for (int t = t0; t < t1;) {
    const int cnt = pre[r + 1] - pre[r], begin = pre[r] * units + unit * cnt, end = begin + cnt;
    const int stop = min(end, t1);
    const int todo = max(0, (stop - t0 - warp + kWarps - 1) / kWarps);  // this warp's tiles up to here
    const int64_t b = a.r0 + r;
    const int hk = unit / a.mtiles, mi = unit - hk * a.mtiles;
    const int h0 = hk * group + mi * C::kRows, rows = min(C::kRows, group - mi * C::kRows);

    if constexpr (kF32) {
      // Scores: lane (key, quarter) takes every fourth 16-byte piece of its key's row. Output: lane owns 4 columns.
      float m[C::kRows], l[C::kRows];  // l: this lane's keys only, quarter 0 counts
      float4 o[C::kRows];
#pragma unroll
      for (int i = 0; i < C::kRows; ++i) m[i] = -INFINITY, l[i] = 0.f, o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      const float* q = static_cast<const float*>(p.q.ptr) + b * p.q.sn + h0 * p.q.sh;
      __syncwarp();
      if (done < todo)
        for (int i = 0; i < rows; ++i)
          if (lane * 4 < p.d)
            *reinterpret_cast<float4*>(q_smem + i * kD + lane * 4) = *reinterpret_cast<const float4*>(q + i * p.q.sh + lane * 4);
      __syncwarp();
      const int key = lane >> 2, quarter = lane & 3, sw = ((key & 1) << 2) | (key >> 1), pieces = p.d >> 2;
      for (; done < todo; ++done) {
        const int stage = done % C::kStages;
        load(done + C::kStages - 1);
        cp_async_wait<C::kStages - 1>();
        __syncwarp();
        const uint8_t* kt = smem + (warp * C::kStages + stage) * C::kStageBytes;
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
#pragma unroll
        for (int j = 0; j < C::kKeys; ++j) {
          const float4 v = *reinterpret_cast<const float4*>(vt + j * C::kRowBytes + ((lane ^ (((j & 1) << 2) | (j >> 1))) << 4));
#pragma unroll
          for (int i = 0; i < C::kRows; ++i) {
            if (i < rows) {
              const float e = p_smem[j * C::kRows + i];
              o[i] = make_float4(fmaf(e, v.x, o[i].x), fmaf(e, v.y, o[i].y), fmaf(e, v.z, o[i].z), fmaf(e, v.w, o[i].w));
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
          if (lane == 0) ml[warp][i] = make_float2(m[i], l[i]);
          if (lane * 4 < p.d) *reinterpret_cast<float4*>(merge + (warp * C::kRows + i) * C::kPitch + lane * 4) = o[i];
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
      if (done < todo) {
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q.ptr) + b * p.q.sn + h0 * p.q.sh;
#pragma unroll
        for (int ks = 0; ks < kD / 16; ++ks)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int i = row + (x & 1) * 8, c = ks * 16 + (x >> 1) * 8 + col;
            qf[ks][x] = i < rows ? *reinterpret_cast<const uint32_t*>(q + i * p.q.sh + c) : 0u;
          }
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
          ldsm4(kt + kr * C::kRowBytes + ((chunk ^ (kr & 7)) << 4), kf);
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
          ldsm4_t(vt + vr * C::kRowBytes + ((chunk ^ (vr & 7)) << 4), vf);
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
        if (i < rows) {
          if ((lane & 3) == 0) ml[warp][i] = make_float2(m[x], l[x]);
          float* to = merge + (warp * C::kRows + i) * C::kPitch + col;
#pragma unroll
          for (int c = 0; c < kD / 8; ++c)
            *reinterpret_cast<float2*>(to + c * 8) = make_float2(o[c][2 * x], o[c][2 * x + 1]);
        }
      }
    }

    // ---- the unit's, or its part's, (O, m, l) out of the four warps' ------------------
    __syncthreads();
    const bool complete = begin >= t0 && end <= t1;
    const int slot = cta * 2 + (begin < t0 ? 0 : 1);
    const int quads = p.d >> 2;
    for (int i = tid; i < rows * quads; i += kThreads) {
      const int row = i / quads, c = (i - row * quads) * 4;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][row].x);
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 x = ml[w][row];
        const float f = ex2_approx(x.x - ref);
        const float4 y = *reinterpret_cast<const float4*>(merge + (w * C::kRows + row) * C::kPitch + c);
        sum = fmaf(f, x.y, sum);
        o = make_float4(fmaf(f, y.x, o.x), fmaf(f, y.y, o.y), fmaf(f, y.z, o.z), fmaf(f, y.w, o.w));
      }
      if (complete) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t at = b * p.out.sn + (h0 + row) * p.out.sh + c;
        if (p.out_is_f32) {
          *reinterpret_cast<float4*>(static_cast<float*>(p.out.ptr) + at) =
              make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        } else {
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out.ptr) + at) =
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
      // the CTA whose run holds the unit's last tile
      int last = (int)(((int64_t)(end - 1) * ctas) / total);
      while ((int64_t)total * (last + 1) / ctas < end) ++last;
      while ((int64_t)total * last / ctas >= end) --last;
      reinterpret_cast<Split*>(ws)[cta] = Split{r, unit, last, 0};
    }
    __syncthreads();
    t = stop;
    if (++unit == units) {
      unit = 0;
      do ++r;
      while (r < a.n && pre[r + 1] == pre[r]);
    }
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
  const int64_t b = a.r0 + sp.b;
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
        int sms = 0, per_sm = 0;
        if ((r = device_sm_count(&sms)) != cudaSuccess) return r;
        r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, paged_decode_kernel<kF32, kD>, kThreads, C::kSmem);
        const int64_t n = (int64_t)sms * (per_sm < 1 ? 1 : per_sm > 2 ? 2 : per_sm);
        *v = n < kMaxCtas ? (int)n : kMaxCtas;
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
  // Requests per launch: their tiles have to stay countable in 31 bits.
  const int64_t per_request = ((keys + C::kKeys - 1) / C::kKeys + 1) * a.units;
  int64_t at_once = per_request > 0 ? ((int64_t(1) << 31) - 1) / per_request : kMaxRequests;
  if (at_once < 1) return cudaErrorInvalidConfiguration;
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
  return ws_layout(16, d <= 64 ? 64 : 128).total > ws_layout(8, 128).total ? ws_layout(16, d <= 64 ? 64 : 128).total
                                                                          : ws_layout(8, 128).total;
}

cudaError_t launch_paged_decode(const PagedDecodeParams& p, cudaStream_t s, int* nlaunch) {
  if (p.is_f32) return launch<true, 128>(p, s, nlaunch);
  return p.d == 64 ? launch<false, 64>(p, s, nlaunch) : launch<false, 128>(p, s, nlaunch);
}

}  // namespace bea
