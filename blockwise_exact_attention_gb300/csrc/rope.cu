// Rotary positions with several axes: every pair (x_p, x_{p + d/2}) of a row
// turned by positions[axis(p)] * freq(p).
//
// The angle. A position is an integer, so only the fractional part of a pair's
// turns per position matters: with T = frac(freq / 2 pi) * 2^64 rounded to an
// integer, position * T in wrapping 64-bit arithmetic is the angle's fraction
// of a turn times 2^64, exact but for T's own rounding. Its upper 32 bits, as
// a signed number, are the angle in half turns times 2^31, which sincospif
// takes; an fp32 angle in radians would be off by 0.004 at position 100000.
//
// HBM-bound: every element is read and written once. A thread owns 16 bytes of
// one half of a row and the 16 bytes of the other half that pair with them; it
// computes their cosines and sines once and turns those pieces of up to
// kHeads heads of its token.
#include <cuda_bf16.h>

#include "launch_cache.cuh"
#include "paged.cuh"

namespace bea {
namespace {

constexpr int kThreads = 128;
constexpr int kHeads = 8;  // heads of one token per thread

template <bool kF32>
struct Piece;  // 16 bytes of a row as fp32 values

template <>
struct Piece<true> {
  static constexpr int kN = 4;
  __device__ static void load(const uint4& r, float* x) {
    x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y), x[2] = __uint_as_float(r.z), x[3] = __uint_as_float(r.w);
  }
  __device__ static uint4 store(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

template <>
struct Piece<false> {
  static constexpr int kN = 8;
  __device__ static void load(const uint4& r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static uint4 store(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <bool kF32>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  using P = Piece<kF32>;
  __shared__ uint64_t turn[kRopeMaxPairs];
  __shared__ uint8_t axis[kRopeMaxPairs];
  const int half = p.d >> 1;
  for (int i = threadIdx.x; i < half; i += kThreads) {
    turn[i] = p.turn[i];
    axis[i] = p.axis[i];
  }
  __syncthreads();
  const int pieces = half / P::kN;  // per half row
  const int heads = p.hq + p.hk;
  const int groups = (heads + kHeads - 1) / kHeads;
  const int64_t total = (int64_t)p.n * p.l * groups * pieces;
  for (int64_t it = (int64_t)blockIdx.x * kThreads + threadIdx.x; it < total; it += (int64_t)gridDim.x * kThreads) {
    const int c = (int)(it % pieces) * P::kN;
    const int64_t tg = it / pieces;
    const int g = (int)(tg % groups);
    const int64_t t = tg / groups;
    const int i = (int)(t % p.l);
    const int64_t b = t / p.l;
    float cs[P::kN], sn[P::kN];
#pragma unroll
    for (int j = 0; j < P::kN; ++j) {
      const int64_t pos = p.pos[axis[c + j] * p.pos_sa + b * p.pos_sn + i];
      const uint64_t a = (uint64_t)pos * turn[c + j];
      sincospif((float)(int32_t)(a >> 32) * 0x1p-31f, &sn[j], &cs[j]);
      if (p.inverse) sn[j] = -sn[j];
    }
    const int h1 = min(heads, (g + 1) * kHeads);
#pragma unroll 4
    for (int hh = g * kHeads; hh < h1; ++hh) {
      const bool isq = hh < p.hq;
      const Seq4& src = isq ? p.q : p.k;
      const Seq4& dst = isq ? p.qo : p.ko;
      const int head = isq ? hh : hh - p.hq;
      constexpr int es = kF32 ? 4 : 2;
      const char* x = static_cast<const char*>(src.ptr) + (b * src.sn + i * src.sl + head * src.sh + c) * es;
      char* y = static_cast<char*>(dst.ptr) + (b * dst.sn + i * dst.sl + head * dst.sh + c) * es;
      float u[P::kN], v[P::kN];
      P::load(*reinterpret_cast<const uint4*>(x), u);
      P::load(*reinterpret_cast<const uint4*>(x + half * es), v);
#pragma unroll
      for (int j = 0; j < P::kN; ++j) {
        const float uj = u[j], vj = v[j];
        u[j] = uj * cs[j] - vj * sn[j];
        v[j] = vj * cs[j] + uj * sn[j];
      }
      *reinterpret_cast<uint4*>(y) = P::store(u);
      *reinterpret_cast<uint4*>(y + half * es) = P::store(v);
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t s, int* nlaunch) {
  const int per = p.is_f32 ? 4 : 8;
  const int groups = (p.hq + p.hk + kHeads - 1) / kHeads;
  const int64_t total = (int64_t)p.n * p.l * groups * (p.d / 2 / per);
  if (total == 0) return cudaSuccess;
  int64_t blocks = (total + kThreads - 1) / kThreads;
  if (blocks > (int64_t(1) << 30)) blocks = int64_t(1) << 30;  // the kernel strides over the rest
  if (p.is_f32)
    rope_kernel<true><<<(unsigned)blocks, kThreads, 0, s>>>(p);
  else
    rope_kernel<false><<<(unsigned)blocks, kThreads, 0, s>>>(p);
  *nlaunch += 1;
  return cudaGetLastError();
}

}  // namespace bea
