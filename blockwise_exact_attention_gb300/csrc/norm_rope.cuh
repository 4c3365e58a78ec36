// Parameter block and launchers of the normed rotary calls, shared by their
// host entry points (rotary_api.cu) and kernels (norm_rope.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "paged.cuh"

namespace bea {

struct NormRopeParams {
  int n, l, hq, hk, d;  // hk = 0: no k
  int pairs;            // turned pairs: the first 2 * pairs elements of a row; the rest passes
  int is_f32, interleaved, norm, inverse;
  float eps, amplitude;
  Seq4 q, k;    // x
  Seq4 gq, gk;  // backward: the gradients of the outputs
  Seq4 qo, ko;  // written: the outputs, or the gradients of x
  const void *wq, *wk;  // [d], or null: ones
  int wq_f32, wk_f32;
  const int32_t* pos;  // [axes, n, l], last dimension contiguous
  int64_t pos_sa, pos_sn;
  // backward: per block and column sums, and the weights' gradients (null: not wanted)
  float* partial;
  void *dwq, *dwk;
  uint64_t turn[kRopeMaxPairs];  // fraction of a turn per position, times 2^64
  uint8_t axis[kRopeMaxPairs];
};
cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t s, int* nlaunch);
size_t norm_rope_bwd_workspace(int64_t d);
cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, cudaStream_t s, int* nlaunch);

}  // namespace bea
