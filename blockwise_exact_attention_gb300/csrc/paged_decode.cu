// Attention of one new token per request over a paged K/V cache.
//
// Online softmax over the request's visible keys, one warp per (request, query
// head): each lane holds 4 elements of the query, of the key it reads and of
// the output.
#include <cuda_bf16.h>

#include "launch_cache.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace bea {
namespace {

constexpr int kWarps = 4;

template <bool kF32>
__device__ __forceinline__ float4 load4(const void* base, int64_t at) {
  if constexpr (kF32) {
    return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
  } else {
    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + at);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xFFFF0000u));
  }
}

template <bool kF32>
__global__ void __launch_bounds__(kWarps * 32) paged_decode_kernel(const __grid_constant__ PagedDecodeParams p) {
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= (int64_t)p.n * p.h) return;
  const int lane = threadIdx.x & 31, hh = (int)(row % p.h), hk = hh / (p.h / p.hkv);
  const int64_t b = row / p.h;
  const bool mine = lane * 4 < p.d;
  int len = p.lens[b];
  const int64_t most = (int64_t)p.max_pages * p.page;
  if (len < 0 || len > most) {
    if (lane == 0) report_status(p.status, BEA_STATUS_PAGES);
    len = len < 0 ? 0 : (int)most;
  }
  const int first = p.left >= len ? 0 : len - 1 - p.left;
  float4 q = make_float4(0.f, 0.f, 0.f, 0.f), o = q;
  if (mine) q = load4<kF32>(p.q.ptr, b * p.q.sn + hh * p.q.sh + lane * 4);
  float m = -INFINITY, l = 0.f;
  const float sl2 = p.scale * 1.4426950408889634f;
  for (int j = first; j < len; ++j) {
    const int pg = j / p.page, off = j - pg * p.page;
    const int id = p.table[b * p.table_stride + pg];
    if (id < 0 || id >= p.num_pages) {
      if (lane == 0) report_status(p.status, BEA_STATUS_PAGES);
      continue;
    }
    float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
    if (mine) {
      k = load4<kF32>(p.kc.ptr, id * p.kc.sn + off * p.kc.sl + hk * p.kc.sh + lane * 4);
      v = load4<kF32>(p.vc.ptr, id * p.vc.sn + off * p.vc.sl + hk * p.vc.sh + lane * 4);
    }
    float s = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    s *= sl2;
    const float mn = fmaxf(m, s);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float w = exp2f(m - ref), e = exp2f(s - ref);
    l = l * w + e;
    o = make_float4(o.x * w + e * v.x, o.y * w + e * v.y, o.z * w + e * v.z, o.w * w + e * v.w);
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (lane == 0) p.lse.ptr[b * p.lse.sn + hh * p.lse.sh] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  if (!mine) return;
  const float r[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
  const int64_t at = b * p.out.sn + hh * p.out.sh + lane * 4;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (p.out_is_f32)
      static_cast<float*>(p.out.ptr)[at + e] = r[e];
    else
      static_cast<__nv_bfloat16*>(p.out.ptr)[at + e] = __float2bfloat16(r[e]);
  }
}

}  // namespace

size_t paged_decode_workspace(int64_t, int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_paged_decode(const PagedDecodeParams& p, cudaStream_t s, int* nlaunch) {
  const int64_t rows = (int64_t)p.n * p.h;
  if (rows == 0) return cudaSuccess;
  const unsigned blocks = (unsigned)((rows + kWarps - 1) / kWarps);
  if (p.is_f32)
    paged_decode_kernel<true><<<blocks, kWarps * 32, 0, s>>>(p);
  else
    paged_decode_kernel<false><<<blocks, kWarps * 32, 0, s>>>(p);
  *nlaunch += 1;
  return cudaGetLastError();
}

}  // namespace bea
