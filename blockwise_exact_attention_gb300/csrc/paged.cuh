// Parameter blocks and launchers of the paged K/V cache calls and of the
// rotary embedding, shared by their host entry points (paged_api.cu) and
// kernels.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"

namespace bea {

// Launch with programmatic stream serialisation: the kernel may be set up while the one before it on the stream still
// runs, so it has to call grid_dependency_wait() in every thread before it touches anything in memory. (The attention
// kernels, whose last writes are bulk copies, let in only the next step of a ring.) A chain of short
// kernels gains 0.4-1 us a launch in a graph, and 1.2 us where the host launches them one by one. Which kernels let the
// next one in early (grid_launch_dependents) is measured: those of one CTA per SM or fewer do, as it hides the next
// one's setup; kernels of many small blocks do not, as the waiting blocks held theirs up (paged_write of 256 tokens in a
// graph 3.0 against 1.6 us, rope_axes 4.7 against 3.0 us).
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// ---- rotary positions ----------------------------------------------------------
constexpr int kRopeMaxPairs = 128;  // d <= 256
constexpr int kRopeMaxAxes = 8;

struct RopeParams {
  int n, l, hq, hk, d;  // hk = 0: no k
  int is_f32, inverse;
  Seq4 q, k, qo, ko;
  const int32_t* pos;  // [axes, n, l], last dimension contiguous
  int64_t pos_sa, pos_sn;
  uint64_t turn[kRopeMaxPairs];  // fraction of a turn per position, times 2^64
  uint8_t axis[kRopeMaxPairs];
};
cudaError_t launch_rope(const RopeParams& p, cudaStream_t s, int* nlaunch);

// ---- paged cache ---------------------------------------------------------------
struct PlanParams {
  int n, max_pages, capacity, n_pool, page;  // n_pool: length of free_pages
  const int32_t *lens, *new_lens, *n_free;
  int32_t* table;
  int64_t table_stride;
  int32_t* pool;
  int32_t *slot_map, *positions, *cu_new, *cu_pages, *lens_out, *n_free_out;
  uint32_t* status;
};
cudaError_t launch_paged_plan(const PlanParams& p, cudaStream_t s, int* nlaunch);

struct PagedWriteParams {
  int n, l, hkv;
  int row_vecs;    // 16-byte pieces per head row
  int es;          // element size in bytes
  int num_slots, page;
  Seq4 k, v;                // [n, l, h_kv, d]
  Seq4 k_cache, v_cache;    // sn: page stride, sl: token stride, sh: head stride
  const int32_t* slot_map;
  uint32_t* status;
};
cudaError_t launch_paged_write(const PagedWriteParams& p, cudaStream_t s, int* nlaunch);

struct PagedDecodeParams {
  int n, h, hkv, d;
  int num_pages, page, max_pages;
  int page_shift;  // log2(page), -1 where page is not a power of two
  int left;        // keys before the last one that are visible (kUnbounded: all)
  int is_f32, out_is_f32;
  float scale;
  Seq4 q, out;  // sl unused (one query per request)
  Seq4 kc, vc;  // sn: page stride, sl: token stride, sh: head stride
  Lse3 lse;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  void* ws;
  uint32_t* status;
};
size_t paged_decode_workspace(int64_t h, int64_t hkv, int64_t d, int64_t max_keys);
// Whether a request's tiles can be counted in 31 bits.
bool paged_decode_fits(int64_t hkv, int64_t d, bool is_f32, int64_t max_keys);
cudaError_t launch_paged_decode(const PagedDecodeParams& p, cudaStream_t s, int* nlaunch);

}  // namespace bea
