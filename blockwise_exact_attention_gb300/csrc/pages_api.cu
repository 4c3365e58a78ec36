// C entry points of the calls on shared pages: argument checks (all before any
// CUDA call) and dispatch.
#include <cstring>

#include "../../include/bea.h"
#include "abi_internal.h"
#include "pages.cuh"

using namespace bea::abi;

namespace {

constexpr int64_t kMost = int64_t(1) << 30;  // of pages, so that sums of two counts fit 32 bits

const int32_t* ints(const bea_tensor* t) { return static_cast<const int32_t*>(t->data); }
int32_t* ints_out(const bea_tensor* t) { return static_cast<int32_t*>(t->data); }

int check_table(const bea_tensor* table, int64_t n, int64_t page_size) {
  int rc;
  if ((rc = check_ints(table, 2))) return rc;
  if (table->shape[0] != n) return BEA_ERR_SHAPE;
  if (page_size < 1 || page_size > (int64_t(1) << 20)) return BEA_ERR_ARG;
  if (table->shape[1] * page_size >= bea::kUnbounded) return BEA_ERR_SHAPE;
  return BEA_OK;
}
// A table that is written: its rows may not overlap.
int check_written_table(const bea_tensor* table) {
  return table->shape[0] > 1 && table->stride[0] < table->shape[1] ? BEA_ERR_ARG : BEA_OK;
}

// The arrays that all these calls have. lens_out, n_free_out: NULL where the call has none.
int check_state(const bea_tensor* lens, const bea_tensor* table, const bea_tensor* shares, const bea_tensor* free_pages,
                const bea_tensor* n_free, int64_t page_size, const bea_tensor* lens_out, const bea_tensor* n_free_out,
                const bea_tensor* shares_out, bea::PagesState* s) {
  int rc;
  for (const bea_tensor* t : {lens, shares, free_pages, n_free, lens_out != nullptr ? lens_out : lens,
                              n_free_out != nullptr ? n_free_out : n_free, shares_out})
    if ((rc = check_ints(t, 1))) return rc;
  const int64_t n = lens->shape[0];
  if ((rc = check_table(table, n, page_size))) return rc;
  if (n_free->shape[0] != 1 || shares_out->shape[0] != shares->shape[0]) return BEA_ERR_SHAPE;
  if (lens_out != nullptr && (lens_out->shape[0] != n || n_free_out->shape[0] != 1)) return BEA_ERR_SHAPE;
  if (shares->shape[0] > kMost || free_pages->shape[0] > kMost) return BEA_ERR_SHAPE;
  s->n = (int)n;
  s->max_pages = (int)table->shape[1];
  s->page = (int)page_size;
  s->n_pool = (int)free_pages->shape[0];
  s->num_pages = (int)shares->shape[0];
  s->lens = ints(lens);
  s->n_free = ints(n_free);
  s->shares = ints(shares);
  s->lens_out = lens_out != nullptr ? ints_out(lens_out) : nullptr;
  s->n_free_out = n_free_out != nullptr ? ints_out(n_free_out) : nullptr;
  s->shares_out = ints_out(shares_out);
  return BEA_OK;
}

// [rows, 3] of copies, without gaps.
int check_copies(const bea_tensor* copies) {
  int rc;
  if ((rc = check_ints(copies, 2))) return rc;
  if (copies->shape[1] != 3) return BEA_ERR_SHAPE;
  return copies->shape[0] > 1 && copies->stride[0] != 3 ? BEA_ERR_ALIGN : BEA_OK;
}

}  // namespace

extern "C" {

int bea_paged_fork(const bea_tensor* src, const bea_tensor* tokens, const bea_tensor* lens,
                   const bea_tensor* block_table, const bea_tensor* shares, const bea_tensor* free_pages,
                   const bea_tensor* n_free, int64_t page_size, const bea_tensor* lens_out,
                   const bea_tensor* n_free_out, const bea_tensor* shares_out, const bea_tensor* copies, void* stream) {
  bea::ForkParams p;
  std::memset(&p, 0, sizeof(p));
  int rc;
  if (lens_out == nullptr || n_free_out == nullptr || block_table == nullptr) return BEA_ERR_ARG;
  if ((rc = check_state(lens, block_table, shares, free_pages, n_free, page_size, lens_out, n_free_out, shares_out, &p.s)))
    return rc;
  if ((rc = check_ints(src, 1)) || (tokens != nullptr && (rc = check_ints(tokens, 1))) || (rc = check_copies(copies)))
    return rc;
  const int64_t n = lens->shape[0];
  if (src->shape[0] != n || (tokens != nullptr && tokens->shape[0] != n) || copies->shape[0] != n) return BEA_ERR_SHAPE;
  if ((rc = check_written_table(block_table))) return rc;
  p.src = ints(src);
  p.tokens = tokens != nullptr ? ints(tokens) : nullptr;
  p.table = ints_out(block_table);
  p.table_stride = block_table->stride[0];
  p.pool = ints(free_pages);
  p.copies = ints_out(copies);
  if ((rc = status_ptr_for_current_device(&p.s.status))) return rc;
  int launches = 0;
  return finish(bea::launch_paged_fork(p, static_cast<cudaStream_t>(stream), &launches), launches);
}

int bea_paged_free(const bea_tensor* ends, const bea_tensor* lens, const bea_tensor* block_table,
                   const bea_tensor* shares, const bea_tensor* free_pages, const bea_tensor* n_free, int64_t page_size,
                   const bea_tensor* lens_out, const bea_tensor* n_free_out, const bea_tensor* shares_out,
                   void* stream) {
  bea::FreeParams p;
  std::memset(&p, 0, sizeof(p));
  int rc;
  if (lens_out == nullptr || n_free_out == nullptr) return BEA_ERR_ARG;
  if ((rc = check_state(lens, block_table, shares, free_pages, n_free, page_size, lens_out, n_free_out, shares_out, &p.s)))
    return rc;
  if ((rc = check_ints(ends, 1))) return rc;
  if (ends->shape[0] != lens->shape[0]) return BEA_ERR_SHAPE;
  p.ends = ints(ends);
  p.table = ints(block_table);
  p.table_stride = block_table->stride[0];
  p.pool = ints_out(free_pages);
  if ((rc = status_ptr_for_current_device(&p.s.status))) return rc;
  int launches = 0;
  return finish(bea::launch_paged_free(p, static_cast<cudaStream_t>(stream), &launches), launches);
}

int bea_paged_compact(const bea_tensor* lens, const bea_tensor* block_table, const bea_tensor* shares,
                      const bea_tensor* free_pages, const bea_tensor* n_free, int64_t page_size,
                      const bea_tensor* block_table_out, const bea_tensor* shares_out, const bea_tensor* free_pages_out,
                      const bea_tensor* page_map, const bea_tensor* copies, void* stream) {
  bea::CompactParams p;
  std::memset(&p, 0, sizeof(p));
  int rc;
  if ((rc = check_state(lens, block_table, shares, free_pages, n_free, page_size, nullptr, nullptr, shares_out, &p.s)))
    return rc;
  if ((rc = check_ints(block_table_out, 2)) || (rc = check_ints(free_pages_out, 1)) || (rc = check_ints(page_map, 1)) ||
      (rc = check_copies(copies)))
    return rc;
  if (!same_shape(block_table_out, block_table) || !same_shape(free_pages_out, free_pages) || !same_shape(page_map, shares))
    return BEA_ERR_SHAPE;
  if ((rc = check_written_table(block_table_out))) return rc;
  if (block_table_out->data == block_table->data && !same_strides(block_table_out, block_table)) return BEA_ERR_ARG;
  if (shares->shape[0] > bea::kCompactMaxPages) return BEA_ERR_UNSUPPORTED;
  if (copies->shape[0] > kMost / 2) return BEA_ERR_SHAPE;
  p.table = ints(block_table);
  p.table_out = ints_out(block_table_out);
  p.table_stride = block_table->stride[0];
  p.table_out_stride = block_table_out->stride[0];
  p.pool = ints(free_pages);
  p.pool_out = ints_out(free_pages_out);
  p.page_map = ints_out(page_map);
  p.copies = ints_out(copies);
  p.capacity = (int)copies->shape[0];
  if ((rc = status_ptr_for_current_device(&p.s.status))) return rc;
  int launches = 0;
  return finish(bea::launch_paged_compact(p, static_cast<cudaStream_t>(stream), &launches), launches);
}

int bea_paged_copy(const bea_tensor* copies, const bea_tensor* caches, int n_caches, void* stream) {
  int rc;
  if (n_caches < 0 || (n_caches > 0 && caches == nullptr)) return BEA_ERR_ARG;
  if ((rc = check_copies(copies))) return rc;
  if (copies->shape[0] > kMost) return BEA_ERR_SHAPE;
  for (int i = 0; i < n_caches; ++i) {
    if ((rc = check_tensor(&caches[i], 4))) return rc;
    if (caches[i].dtype != caches[0].dtype) return BEA_ERR_DTYPE;
    if (!same_shape(&caches[i], &caches[0])) return BEA_ERR_SHAPE;
    if (broadcast(&caches[i])) return BEA_ERR_ARG;
  }
  if (n_caches == 0) return finish(cudaSuccess, 0);
  const int64_t *shape = caches[0].shape, es = caches[0].dtype == BEA_F32 ? 4 : 2, row = shape[3] * es;
  if (row % 16 != 0) return BEA_ERR_UNSUPPORTED;
  if (shape[1] > kMost || shape[2] > kMost || row > kMost || shape[1] * shape[2] > kMost ||
      shape[1] * shape[2] * (row / 16) > kMost)
    return BEA_ERR_SHAPE;
  if (copies->shape[0] == 0 || shape[0] == 0 || shape[1] == 0 || shape[2] == 0 || shape[3] == 0)
    return finish(cudaSuccess, 0);
  bea::CopyParams p;
  std::memset(&p, 0, sizeof(p));
  p.m = (int)copies->shape[0];
  p.num_pages = (int)shape[0];
  p.page = (int)shape[1];
  p.hkv = (int)shape[2];
  p.row_vecs = (int)(row / 16);
  p.chunks = bea::copy_chunks(p.page, p.hkv, p.row_vecs);
  p.copies = ints(copies);
  if ((rc = status_ptr_for_current_device(&p.status))) return rc;
  int launches = 0;
  cudaError_t e = cudaSuccess;
  for (int i0 = 0; i0 < n_caches && e == cudaSuccess; i0 += bea::kCopyCaches) {
    p.n_caches = n_caches - i0 < bea::kCopyCaches ? n_caches - i0 : bea::kCopyCaches;
    for (int i = 0; i < p.n_caches; ++i) {
      const bea_tensor& c = caches[i0 + i];
      auto& to = p.cache[i];
      to.ptr = static_cast<char*>(c.data);
      to.sn = c.stride[0] * es;
      to.sl = c.stride[1] * es;
      to.sh = c.stride[2] * es;
      const bool heads = shape[2] == 1 || to.sh == row, dense = heads && (shape[1] == 1 || to.sl == shape[2] * row);
      if (dense) to.sl = 0;
      else if (to.sl == 0) to.sl = 16;  // one token: not used, and not the mark of a dense page
    }
    e = bea::launch_paged_copy(p, static_cast<cudaStream_t>(stream), &launches);
  }
  return finish(e, launches);
}

}  // extern "C"
