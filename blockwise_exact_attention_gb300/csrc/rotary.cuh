// What the rotary kernels share: 16-byte pieces of a row as fp32 values, and the
// cosine and sine of a position times a frequency (rope.cu says why they are
// computed this way).
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

namespace bea {

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

// `turn`: the frequency as the fraction of a turn per position, times 2^64.
__device__ __forceinline__ void cos_sin(int64_t pos, uint64_t turn, int inverse, float* cs, float* sn) {
  const uint64_t a = (uint64_t)pos * turn;
  const uint32_t quarter = ((uint32_t)(a >> 32) + 0x20000000u) >> 30;  // the nearest; bit 61 of a is the rest's sign
  float s, x;
  sincospif((float)(int32_t)(a >> 30) * 0x1p-33f, &s, &x);
  *cs = quarter & 1u ? s : x;
  *sn = quarter & 1u ? x : s;
  if ((quarter + 1u) & 2u) *cs = -*cs;
  if (((quarter >> 1) & 1u) != (uint32_t)inverse) *sn = -*sn;
}

}  // namespace bea
