// RMS norm of every head of q and k, then the rotation, in one pass; and its gradient.
//
// A row x of d elements becomes y = w * x * r, r = 1 / sqrt(mean(x^2) + eps), and y's first 2 * pairs elements are
// turned pair by pair, (a, b) -> (a c - b s, b c + a s), with c and s the angle's cosine and sine times the amplitude.
// Pairs are (x_p, x_{p + pairs}) or, interleaved, (x_{2p}, x_{2p + 1}); what lies behind passes. Without the norm it is
// the rotation alone. All of it in fp32, one rounding at the end. With g the gradient turned back (the rotation's
// adjoint), the gradients are
//   dw = sum over rows of g * x r,   dx = r (w g - x r^2 mean(w g x)).
//
// HBM-bound: forward 2 elements moved for one of x, backward 3. A row belongs to `lanes` neighbouring lanes of a warp, a
// power of two; each holds two 16-byte pieces of it, both ends of its pairs (half layout: a piece of the first half and its
// partner in the second; interleaved: 32 bytes in a row), so the rotation needs no exchange and the norm a shuffle tree
// of log2(lanes) steps. A thread does kHeads heads of one token: it sends their loads, works out the cosines and sines
// while they are under way, then reduces, turns and stores.
//
// The weights' gradient is a sum over all rows. A thread keeps its columns' sums in fp32 over all the rows it meets
// (the grid is one wave, each block only q or only k), a block adds up its threads in shared memory, and a second kernel
// the blocks, all in a fixed order: the same call gives the same bits.
#include <type_traits>

#include <cuda_bf16.h>

#include "launch_cache.cuh"
#include "norm_rope.cuh"
#include "ptx.cuh"
#include "rotary.cuh"

namespace bea {
namespace {

constexpr int kThreads = 128;
constexpr int kSmThreads = 2048;  // that an SM holds
constexpr int kMaxD = 2 * kRopeMaxPairs;

__device__ __forceinline__ float weight_at(const void* w, int is_f32, int c) {
  if (w == nullptr) return 1.f;
  return is_f32 ? static_cast<const float*>(w)[c] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c]);
}

// Where lane `i` of a row finds its two pieces (of N elements): columns a and b, and its pairs: i * N + j, j < N.
template <bool kInter, int N>
struct Place {
  int a, b, pair;
  bool mine;
  __device__ __forceinline__ Place(int i, int d, int pairs) {
    pair = i * N;
    mine = 2 * i * N < d;
    if (kInter) {
      a = 2 * i * N;
      b = a + N;
    } else if (pair < pairs) {  // pairs is a multiple of N
      a = pair;
      b = pair + pairs;
    } else {
      a = 2 * i * N;
      b = a + N;
    }
  }
  // The column of the first and second element of pair j.
  __device__ __forceinline__ int first(int j) const { return kInter ? a + 2 * j : a + j; }
  __device__ __forceinline__ int second(int j) const { return kInter ? a + 2 * j + 1 : b + j; }
};

// The pieces of a row as the first and second elements of its pairs, and back.
template <bool kF32, bool kInter>
__device__ __forceinline__ void unpack(const uint4& ra, const uint4& rb, float* u, float* v) {
  using P = Piece<kF32>;
  if constexpr (!kInter) {
    P::load(ra, u);
    P::load(rb, v);
  } else {
    float x[2 * P::kN];
    P::load(ra, x);
    P::load(rb, x + P::kN);
#pragma unroll
    for (int j = 0; j < P::kN; ++j) u[j] = x[2 * j], v[j] = x[2 * j + 1];
  }
}
template <bool kF32, bool kInter>
__device__ __forceinline__ void pack(const float* u, const float* v, uint4& ra, uint4& rb) {
  using P = Piece<kF32>;
  if constexpr (!kInter) {
    ra = P::store(u);
    rb = P::store(v);
  } else {
    float x[2 * P::kN];
#pragma unroll
    for (int j = 0; j < P::kN; ++j) x[2 * j] = u[j], x[2 * j + 1] = v[j];
    ra = P::store(x);
    rb = P::store(x + P::kN);
  }
}

// Turns the pairs that are turned; the others pass untouched, whatever they hold.
template <int N>
__device__ __forceinline__ void turn_pairs(float* u, float* v, const float* cs, const float* sn, int pair, int pairs) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float a = u[j], b = v[j];
    if (pair + j < pairs) {
      u[j] = a * cs[j] - b * sn[j];
      v[j] = b * cs[j] + a * sn[j];
    }
  }
}

struct Tables {
  uint64_t turn[kRopeMaxPairs];
  uint8_t axis[kRopeMaxPairs];
  float w[2][kMaxD];
};
// Those of the launch before the wait on the kernel before, the weights after it.
template <bool kNorm>
__device__ __forceinline__ void load_tables(const NormRopeParams& p, Tables& t) {
  for (int i = threadIdx.x; i < p.pairs; i += blockDim.x) {
    t.turn[i] = p.turn[i];
    t.axis[i] = p.axis[i];
  }
  grid_dependency_wait();
  if constexpr (kNorm) {
    for (int i = threadIdx.x; i < p.d; i += blockDim.x) {
      t.w[0][i] = weight_at(p.wq, p.wq_f32, i);
      t.w[1][i] = weight_at(p.wk, p.wk_f32, i);
    }
  }
  __syncthreads();
}

template <int N>
__device__ __forceinline__ void angles(const NormRopeParams& p, const Tables& t, int64_t b, int i, int pair, int inverse,
                                       float* cs, float* sn) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    cs[j] = 1.f, sn[j] = 0.f;
    if (pair + j < p.pairs) {
      const int64_t pos = p.pos[t.axis[pair + j] * p.pos_sa + b * p.pos_sn + i];
      cos_sin(pos, t.turn[pair + j], inverse, &cs[j], &sn[j]);
      cs[j] *= p.amplitude;
      sn[j] *= p.amplitude;
    }
  }
}

__device__ __forceinline__ int lane_shift(int d, int n) {  // lanes of a row: half its pieces, up to a power of two
  const int half = (d / n + 1) / 2;
  return half <= 1 ? 0 : 32 - __clz(half - 1);
}
int host_lane_shift(int d, int n) {
  int s = 0;
  while ((1 << s) * 2 * n < d) ++s;
  return s;
}

// Index: of a lane's work item; 32 bits where they are enough.
template <bool kF32, bool kNorm, bool kInter, int kHeads, typename Index>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  using P = Piece<kF32>;
  constexpr int N = P::kN;
  __shared__ Tables tables;
  load_tables<kNorm>(p, tables);
  constexpr int es = kF32 ? 4 : 2;
  const int shift = lane_shift(p.d, N), lane = threadIdx.x & ((1 << shift) - 1);
  const Place<kInter, N> at(lane, p.d, p.pairs);
  const unsigned gq = (p.hq + kHeads - 1) / kHeads, groups = gq + (p.hk + kHeads - 1) / kHeads;
  const Index total = ((Index)p.n * p.l * groups) << shift;
  const float inv_d = 1.f / (float)p.d;
  // a warp goes on while any of its items is one, so that all its lanes meet in the shuffles
  for (Index it = (Index)blockIdx.x * kThreads + threadIdx.x; (it & ~(Index)31) < total; it += (Index)gridDim.x * kThreads) {
    const bool live = it < total && at.mine;
    const Index tg = live ? it >> shift : 0, t = tg / groups;
    const unsigned g = (unsigned)(tg - t * groups);
    const bool is_k = g >= gq;
    const int h0 = (int)(is_k ? g - gq : g) * kHeads, heads = is_k ? p.hk : p.hq;
    const int64_t b = t / p.l;
    const int i = (int)(t - (Index)b * p.l);
    const Seq4 &from = is_k ? p.k : p.q, &to = is_k ? p.ko : p.qo;
    uint4 ra[kHeads], rb[kHeads];
    const char* src = static_cast<const char*>(from.ptr) + (b * from.sn + i * from.sl + h0 * from.sh) * es;
#pragma unroll
    for (int x = 0; x < kHeads; ++x) {
      ra[x] = rb[x] = make_uint4(0u, 0u, 0u, 0u);
      if (live && h0 + x < heads) {
        ra[x] = __ldcs(reinterpret_cast<const uint4*>(src + (x * from.sh + at.a) * es));
        rb[x] = __ldcs(reinterpret_cast<const uint4*>(src + (x * from.sh + at.b) * es));
      }
    }
    float cs[N], sn[N];
    angles<N>(p, tables, b, i, at.mine ? at.pair : p.pairs, p.inverse, cs, sn);
    char* dst = static_cast<char*>(to.ptr) + (b * to.sn + i * to.sl + h0 * to.sh) * es;
#pragma unroll
    for (int x = 0; x < kHeads; ++x) {
      float u[N], v[N];
      unpack<kF32, kInter>(ra[x], rb[x], u, v);
      if constexpr (kNorm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) ss = fmaf(u[j], u[j], fmaf(v[j], v[j], ss));
        for (int o = 1; o < (1 << shift); o <<= 1) ss += __shfl_xor_sync(~0u, ss, o);
        const float r = __frsqrt_rn(fmaf(ss, inv_d, p.eps));
        const float* w = tables.w[is_k];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          u[j] *= r * (at.mine ? w[at.first(j)] : 0.f);
          v[j] *= r * (at.mine ? w[at.second(j)] : 0.f);
        }
      }
      turn_pairs<N>(u, v, cs, sn, at.pair, p.pairs);
      if (live && h0 + x < heads) {
        uint4 oa, ob;
        pack<kF32, kInter>(u, v, oa, ob);
        uint4 *pa = reinterpret_cast<uint4*>(dst + (x * to.sh + at.a) * es),
              *pb = reinterpret_cast<uint4*>(dst + (x * to.sh + at.b) * es);
        if constexpr (kHeads == 8) {
          __stcs(pa, oa);
          __stcs(pb, ob);
        } else {
          *pa = oa;
          *pb = ob;
        }
      }
    }
  }
}

// The gradient under the norm. Blocks [0, bq) do q, the others k; a block's threads step over its part's items.
template <bool kF32, bool kInter, int kHeads>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p, int bq) {
  using P = Piece<kF32>;
  constexpr int N = P::kN;
  __shared__ Tables tables;
  __shared__ float sums[kThreads * 2 * N];
  load_tables<true>(p, tables);
  constexpr int es = kF32 ? 4 : 2;
  const int shift = lane_shift(p.d, N), lane = threadIdx.x & ((1 << shift) - 1);
  const Place<kInter, N> at(lane, p.d, p.pairs);
  const bool is_k = (int)blockIdx.x >= bq;
  const int64_t block = is_k ? blockIdx.x - bq : blockIdx.x, blocks = is_k ? gridDim.x - bq : bq;
  const int heads = is_k ? p.hk : p.hq;
  const Seq4 &from = is_k ? p.k : p.q, &grad = is_k ? p.gk : p.gq, &to = is_k ? p.ko : p.qo;
  const unsigned groups = (heads + kHeads - 1) / kHeads;
  const int64_t total = ((int64_t)p.n * p.l * groups) << shift;
  const float inv_d = 1.f / (float)p.d;
  float wa[N], wb[N], da[N], db[N];  // weights and their gradients' sums, of this lane's pairs
#pragma unroll
  for (int j = 0; j < N; ++j) {
    wa[j] = at.mine ? tables.w[is_k][at.first(j)] : 0.f;
    wb[j] = at.mine ? tables.w[is_k][at.second(j)] : 0.f;
    da[j] = db[j] = 0.f;
  }
  for (int64_t it = block * kThreads + threadIdx.x; (it & ~int64_t(31)) < total; it += blocks * kThreads) {
    const bool live = it < total && at.mine;
    const int64_t tg = live ? it >> shift : 0;
    int64_t t, b;
    if (total < (int64_t(1) << 31)) {
      t = (uint32_t)tg / groups;
      b = (uint32_t)t / (uint32_t)p.l;
    } else {
      t = tg / groups;
      b = t / p.l;
    }
    const int h0 = (int)(tg - t * groups) * kHeads, i = (int)(t - b * p.l);
    const char* src = static_cast<const char*>(from.ptr) + (b * from.sn + i * from.sl + h0 * from.sh) * es;
    const char* gsrc = static_cast<const char*>(grad.ptr) + (b * grad.sn + i * grad.sl + h0 * grad.sh) * es;
    uint4 ra[kHeads], rb[kHeads], ga[kHeads], gb[kHeads];
#pragma unroll
    for (int x = 0; x < kHeads; ++x) {
      ra[x] = rb[x] = ga[x] = gb[x] = make_uint4(0u, 0u, 0u, 0u);
      if (live && h0 + x < heads) {
        ra[x] = __ldcs(reinterpret_cast<const uint4*>(src + (x * from.sh + at.a) * es));
        rb[x] = __ldcs(reinterpret_cast<const uint4*>(src + (x * from.sh + at.b) * es));
        ga[x] = __ldcs(reinterpret_cast<const uint4*>(gsrc + (x * grad.sh + at.a) * es));
        gb[x] = __ldcs(reinterpret_cast<const uint4*>(gsrc + (x * grad.sh + at.b) * es));
      }
    }
    float cs[N], sn[N];
    angles<N>(p, tables, b, i, at.mine ? at.pair : p.pairs, 1, cs, sn);
    char* dst = static_cast<char*>(to.ptr) + (b * to.sn + i * to.sl + h0 * to.sh) * es;
#pragma unroll
    for (int x = 0; x < kHeads; ++x) {
      float u[N], v[N], gu[N], gv[N];
      unpack<kF32, kInter>(ra[x], rb[x], u, v);
      unpack<kF32, kInter>(ga[x], gb[x], gu, gv);
      turn_pairs<N>(gu, gv, cs, sn, at.pair, p.pairs);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        ss = fmaf(u[j], u[j], fmaf(v[j], v[j], ss));
        dot = fmaf(gu[j] * wa[j], u[j], fmaf(gv[j] * wb[j], v[j], dot));
      }
      for (int o = 1; o < (1 << shift); o <<= 1) {
        ss += __shfl_xor_sync(~0u, ss, o);
        dot += __shfl_xor_sync(~0u, dot, o);
      }
      if (!(live && h0 + x < heads)) continue;
      const float r = __frsqrt_rn(fmaf(ss, inv_d, p.eps)), c = dot * inv_d * r * r;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        da[j] = fmaf(gu[j], u[j] * r, da[j]);
        db[j] = fmaf(gv[j], v[j] * r, db[j]);
        u[j] = r * (gu[j] * wa[j] - u[j] * c);
        v[j] = r * (gv[j] * wb[j] - v[j] * c);
      }
      uint4 oa, ob;
      pack<kF32, kInter>(u, v, oa, ob);
      __stcs(reinterpret_cast<uint4*>(dst + (x * to.sh + at.a) * es), oa);
      __stcs(reinterpret_cast<uint4*>(dst + (x * to.sh + at.b) * es), ob);
    }
  }
  if ((is_k ? p.dwk : p.dwq) == nullptr) return;
  // rows of d: one of every group of lanes
  if (at.mine) {
    float* row = sums + (threadIdx.x >> shift) * p.d;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      row[at.first(j)] = da[j];
      row[at.second(j)] = db[j];
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < p.d; c += kThreads) {
    float s = 0.f;
    for (int r = 0; r < (kThreads >> shift); ++r) s += sums[r * p.d + c];
    p.partial[(int64_t)blockIdx.x * p.d + c] = s;
  }
}

// The blocks' sums, 32 columns a block, a warp every kSumWarps-th of them.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32) norm_rope_weight_kernel(const __grid_constant__ NormRopeParams p, int bq, int blocks) {
  __shared__ float part[kSumWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, is_k = blockIdx.y;
  grid_dependency_wait();
  void* out = is_k ? p.dwk : p.dwq;
  if (out == nullptr) return;
  const int b0 = is_k ? bq : 0, b1 = is_k ? blocks : bq;
  float s = 0.f;
  if (c < p.d) {
#pragma unroll 8
    for (int b = b0 + warp; b < b1; b += kSumWarps) s += p.partial[(int64_t)b * p.d + c];
  }
  part[warp][lane] = s;
  __syncthreads();
  s = part[lane][warp];  // column blockIdx.x * 32 + warp, part `lane`
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  const int col = blockIdx.x * 32 + warp;
  if (lane == 0 && col < p.d) {
    if (is_k ? p.wk_f32 : p.wq_f32)
      static_cast<float*>(out)[col] = s;
    else
      static_cast<__nv_bfloat16*>(out)[col] = __float2bfloat16(s);
  }
}

// A runtime truth value as a type.
template <typename F>
auto with(bool x, F f) {
  return x ? f(std::true_type{}) : f(std::false_type{});
}

template <bool kF32, bool kNorm, bool kInter>
cudaError_t launch_fwd(const NormRopeParams& p, cudaStream_t s) {
  constexpr int N = kF32 ? 4 : 8;
  const int shift = host_lane_shift(p.d, N);
  auto items = [&](int heads) {
    return ((int64_t)p.n * p.l * ((p.hq + heads - 1) / heads + (p.hk + heads - 1) / heads)) << shift;
  };
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const bool wide = items(8) >= (int64_t)sms * kSmThreads;  // enough to fill the GPU
  int64_t blocks = (items(wide ? 8 : 4) + kThreads - 1) / kThreads;
  if (blocks > (int64_t(1) << 30)) blocks = int64_t(1) << 30;  // the kernel strides over the rest
  const bool narrow = blocks * kThreads * 2 < (int64_t(1) << 32);
  auto kern = wide ? (narrow ? norm_rope_kernel<kF32, kNorm, kInter, 8, uint32_t> : norm_rope_kernel<kF32, kNorm, kInter, 8, uint64_t>)
                   : norm_rope_kernel<kF32, kNorm, kInter, 4, uint32_t>;  // not wide: few items
  return launch_dependent(kern, dim3((unsigned)blocks), kThreads, 0, s, p);
}

constexpr int kBwdHeads = 4;
constexpr int kBwdMaxBlocks = 2048;

template <bool kF32, bool kInter>
cudaError_t launch_bwd(const NormRopeParams& p, cudaStream_t s, int* bq, int* blocks) {
  constexpr int N = kF32 ? 4 : 8;
  static PerContext<int> cache;
  int cap = 0;
  cudaError_t e = wave_cap(cache, norm_rope_bwd_kernel<kF32, kInter, kBwdHeads>, kThreads, 0, &cap);
  if (e != cudaSuccess) return e;
  if (cap > kBwdMaxBlocks) cap = kBwdMaxBlocks;
  const int shift = host_lane_shift(p.d, N);
  auto need = [&](int heads) {
    return ((((int64_t)p.n * p.l * ((heads + kBwdHeads - 1) / kBwdHeads)) << shift) + kThreads - 1) / kThreads;
  };
  const int64_t q = need(p.hq), k = need(p.hk);
  // a wave shared out by work, at least a block for each that has some
  int64_t nq = q, nk = k;
  if (q + k > cap) {
    nq = k == 0 ? cap : (int64_t)((double)cap * q / (double)(q + k) + 0.5);
    if (nq < 1) nq = 1;
    if (k > 0 && nq > cap - 1) nq = cap - 1;
    nk = cap - nq;
    if (nk > k) nk = k;
    if (nq > q) nq = q;
  }
  *bq = (int)nq;
  *blocks = (int)(nq + nk);
  if (*blocks == 0) return cudaSuccess;
  return launch_dependent(norm_rope_bwd_kernel<kF32, kInter, kBwdHeads>, dim3((unsigned)*blocks), kThreads, 0, s, p, *bq);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t s, int* nlaunch) {
  const cudaError_t e = with(p.is_f32, [&](auto f32) {
    return with(p.norm, [&](auto norm) {
      return with(p.interleaved, [&](auto inter) {
        return launch_fwd<decltype(f32)::value, decltype(norm)::value, decltype(inter)::value>(p, s);
      });
    });
  });
  if (e == cudaSuccess) *nlaunch += 1;
  return e;
}

size_t norm_rope_bwd_workspace(int64_t d) { return (size_t)kBwdMaxBlocks * (size_t)d * 4; }

cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, cudaStream_t s, int* nlaunch) {
  int bq = 0, blocks = 0;
  cudaError_t e = with(p.is_f32, [&](auto f32) {
    return with(p.interleaved, [&](auto inter) {
      return launch_bwd<decltype(f32)::value, decltype(inter)::value>(p, s, &bq, &blocks);
    });
  });
  if (e != cudaSuccess) return e;
  if (blocks > 0) *nlaunch += 1;
  if (p.dwq == nullptr && p.dwk == nullptr) return e;
  e = launch_dependent(norm_rope_weight_kernel, dim3((unsigned)((p.d + 31) / 32), 2), kSumWarps * 32, 0, s, p, bq, blocks);
  if (e == cudaSuccess) *nlaunch += 1;
  return e;
}

}  // namespace bea
