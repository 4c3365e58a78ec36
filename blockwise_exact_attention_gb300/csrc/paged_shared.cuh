// Parameter block and launcher of attention over a shared prefix, shared by its
// host entry point (shared_api.cu) and kernels (paged_shared.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "paged.cuh"

namespace bea {

constexpr int kMaxGroups = 1024;  // their schedule is scanned in shared memory

struct PagedSharedParams {
  PagedDecodeParams d;  // ws: the whole workspace
  int groups;
  const int32_t *group_rows, *shared_lens;
};
// Whether sharing could save so little, by the table's width, that paged_decode is faster for all.
bool paged_shared_is_plain(const PagedDecodeParams& d, int64_t groups);
size_t paged_shared_workspace(int64_t n, int64_t h, int64_t h_kv, int64_t d, int64_t max_keys, int64_t groups);
// Whether the counts of the schedule fit 31 bits.
bool paged_shared_fits(int64_t n, int64_t h, int64_t h_kv, int64_t max_keys, int64_t groups);
// Of a page's rows tiles of 128 take any multiple of the largest power of two, up to 128, that divides a page.
int paged_shared_box(int64_t page);
// Boxes of 64 columns and paged_shared_box(page) << i tokens, those of no more than a page and a tile.
constexpr int kPageMaps = 8;
struct PageMaps {
  CUtensorMap k[kPageMaps], v[kPageMaps];
};
cudaError_t launch_paged_shared(const PagedSharedParams& p, const PageMaps& maps, cudaStream_t s, int* nlaunch);

}  // namespace bea
