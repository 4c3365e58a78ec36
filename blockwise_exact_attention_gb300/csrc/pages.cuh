// Parameter blocks and launchers of the calls on shared pages (fork, free,
// compact, copy), shared by their host entry points (pages_api.cu) and kernels
// (pages.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"

namespace bea {

// What the calls on tables have in common. An output may be its input.
struct PagesState {
  int n, max_pages, page, n_pool, num_pages;  // n_pool: length of free_pages; num_pages: of shares
  const int32_t *lens, *n_free, *shares;
  int32_t *lens_out, *n_free_out, *shares_out;
  uint32_t* status;
};

struct ForkParams {
  PagesState s;
  const int32_t *src, *tokens;  // tokens null: all of the source's
  int32_t* table;
  int64_t table_stride;
  const int32_t* pool;
  int32_t* copies;  // [n, 3]
};
cudaError_t launch_paged_fork(const ForkParams& p, cudaStream_t s, int* nlaunch);

struct FreeParams {
  PagesState s;
  const int32_t* ends;
  const int32_t* table;
  int64_t table_stride;
  int32_t* pool;
};
cudaError_t launch_paged_free(const FreeParams& p, cudaStream_t s, int* nlaunch);

constexpr int kCompactMaxPages = 1 << 20;  // a bit of shared memory each
struct CompactParams {
  PagesState s;  // lens_out, n_free_out unused
  const int32_t* table;
  int32_t* table_out;
  int64_t table_stride, table_out_stride;
  const int32_t* pool;
  int32_t* pool_out;
  int32_t *page_map, *copies;
  int capacity;
};
cudaError_t launch_paged_compact(const CompactParams& p, cudaStream_t s, int* nlaunch);

constexpr int kCopyCaches = 64;  // per launch
struct CopyParams {
  int m, n_caches, num_pages, page, hkv;
  int row_vecs;    // 16-byte pieces of a head's row
  int chunks;      // of a page
  const int32_t* copies;  // [m, 3]
  struct Cache {
    char* ptr;
    int64_t sn, sl, sh;  // bytes; sl = 0: a page's tokens and heads lie one behind the other
  } cache[kCopyCaches];
  uint32_t* status;
};
cudaError_t launch_paged_copy(CopyParams& p, cudaStream_t s, int* nlaunch);
int copy_chunks(int64_t page, int64_t hkv, int64_t row_vecs);

}  // namespace bea
