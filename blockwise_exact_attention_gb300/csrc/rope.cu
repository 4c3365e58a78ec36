// Rotary positions with several axes: every pair (x_p, x_{p + d/2}) of a row
// turned by positions[axis(p)] * freq(p).
//
// The angle. A position is an integer, so only the fractional part of a pair's
// turns per position matters: with T = frac(freq / 2 pi) * 2^64 rounded to an
// integer, position * T in wrapping 64-bit arithmetic is the angle's fraction
// of a turn times 2^64, exact but for T's own rounding. Its upper bits give the
// nearest quarter turn, which only swaps and negates; the rest, at most a quarter
// of a half turn, goes to sincospif in fp32 and is off by 2^-27 half turns at
// most. (The whole angle in fp32 half turns: 2^-25, cosines and sines up to
// 1.1e-7 off instead of 8e-8; an fp32 angle in radians would be off by 0.004 at
// position 100000.)
//
// HBM-bound: every element is read and written once. A thread owns 16 bytes of
// one half of a row and the 16 bytes of the other half that pair with them, in
// kHeads heads of one token: it sends all its loads, computes the pieces'
// cosines and sines while they are under way, turns and stores. With 8 heads the
// cosines and sines cost half as much and the stores are streamed past L2: 206 us
// for forward and gradient of [1, 32768, 32 + 8, 128] bf16 against 229 us with 4
// (now 203 us, 6.6 TB/s). Where 8 heads would leave the GPU's threads unfilled it
// takes 4: 17.0 against 22.4 us for [3, 1369, 12 + 12, 64] f32 (now 17.3 us), 4.3
// against 5.5 us for 256 tokens of 32 + 8 heads (now 3.0 us).
#include <type_traits>

#include "launch_cache.cuh"
#include "paged.cuh"
#include "ptx.cuh"
#include "rotary.cuh"

namespace bea {
namespace {

constexpr int kThreads = 128;
constexpr int kSmThreads = 2048;  // that an SM holds

// Index: of a thread's work item; 32 bits where they are enough, three divisions by run-time numbers start each item.
template <bool kF32, int kHeads, typename Index>
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
  grid_dependency_wait();
  constexpr int es = kF32 ? 4 : 2;
  const unsigned pieces = half / P::kN;  // per half row
  const int heads = p.hq + p.hk;
  const unsigned groups = (heads + kHeads - 1) / kHeads;
  const Index total = (Index)p.n * p.l * groups * pieces;
  for (Index it = (Index)blockIdx.x * kThreads + threadIdx.x; it < total; it += (Index)gridDim.x * kThreads) {
    const Index tg = it / pieces, t = tg / groups;
    const int c = (int)(it - tg * pieces) * P::kN;
    const int first = (int)(tg - t * groups) * kHeads;
    const int64_t b = t / p.l;
    const int i = (int)(t - (Index)b * p.l);
    uint4 ru[kHeads], rv[kHeads];
#pragma unroll
    for (int x = 0; x < kHeads; ++x) {
      const int hh = first + x;
      if (hh >= heads) continue;
      const char* base = hh < p.hq ? static_cast<const char*>(p.q.ptr) + (b * p.q.sn + i * p.q.sl + hh * p.q.sh + c) * es
                                   : static_cast<const char*>(p.k.ptr) +
                                         (b * p.k.sn + i * p.k.sl + (hh - p.hq) * p.k.sh + c) * es;
      ru[x] = __ldcs(reinterpret_cast<const uint4*>(base));
      rv[x] = __ldcs(reinterpret_cast<const uint4*>(base + half * es));
    }
    float cs[P::kN], sn[P::kN];
#pragma unroll
    for (int j = 0; j < P::kN; ++j) {
      const int64_t pos = p.pos[axis[c + j] * p.pos_sa + b * p.pos_sn + i];
      cos_sin(pos, turn[c + j], p.inverse, &cs[j], &sn[j]);
    }
#pragma unroll
    for (int x = 0; x < kHeads; ++x) {
      const int hh = first + x;
      if (hh >= heads) continue;
      char* base = hh < p.hq ? static_cast<char*>(p.qo.ptr) + (b * p.qo.sn + i * p.qo.sl + hh * p.qo.sh + c) * es
                             : static_cast<char*>(p.ko.ptr) +
                                   (b * p.ko.sn + i * p.ko.sl + (hh - p.hq) * p.ko.sh + c) * es;
      float u[P::kN], v[P::kN];
      P::load(ru[x], u);
      P::load(rv[x], v);
#pragma unroll
      for (int j = 0; j < P::kN; ++j) {
        const float uj = u[j], vj = v[j];
        u[j] = uj * cs[j] - vj * sn[j];
        v[j] = vj * cs[j] + uj * sn[j];
      }
      if constexpr (kHeads == 8) {
        __stcs(reinterpret_cast<uint4*>(base), P::store(u));
        __stcs(reinterpret_cast<uint4*>(base + half * es), P::store(v));
      } else {
        *reinterpret_cast<uint4*>(base) = P::store(u);
        *reinterpret_cast<uint4*>(base + half * es) = P::store(v);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t s, int* nlaunch) {
  const int64_t pieces = p.d / 2 / (p.is_f32 ? 4 : 8), tokens = (int64_t)p.n * p.l;
  auto threads = [&](int heads) { return tokens * ((p.hq + p.hk + heads - 1) / heads) * pieces; };
  if (threads(1) == 0) return cudaSuccess;
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const bool wide = threads(8) >= (int64_t)sms * kSmThreads;  // enough to fill the GPU
  const int64_t total = threads(wide ? 8 : 4);
  int64_t blocks = (total + kThreads - 1) / kThreads;
  if (blocks > (int64_t(1) << 30)) blocks = int64_t(1) << 30;  // the kernel strides over the rest
  const bool narrow = blocks * kThreads * 2 < (int64_t(1) << 32);
  auto pick = [&](auto f32, auto heads) {
    constexpr bool kF32 = decltype(f32)::value;
    constexpr int kHeads = decltype(heads)::value;
    return narrow ? rope_kernel<kF32, kHeads, uint32_t> : rope_kernel<kF32, kHeads, uint64_t>;
  };
  using Four = std::integral_constant<int, 4>;
  using Eight = std::integral_constant<int, 8>;
  auto kern = p.is_f32 ? (wide ? pick(std::true_type{}, Eight{}) : pick(std::true_type{}, Four{}))
                       : (wide ? pick(std::false_type{}, Eight{}) : pick(std::false_type{}, Four{}));
  e = launch_dependent(kern, dim3((unsigned)blocks), kThreads, 0, s, p);
  if (e == cudaSuccess) *nlaunch += 1;
  return e;
}

}  // namespace bea
