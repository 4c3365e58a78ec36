// C entry points of the rotary embedding and the paged K/V cache: argument
// checks (all before any CUDA call) and dispatch.
#include <cmath>
#include <cstring>

#include "../../include/bea.h"
#include "abi_internal.h"
#include "paged.cuh"

namespace bea {
namespace abi {

// An i32 tensor: rank, dtype, non-negative shape and strides, contiguous last
// dimension, 4-byte aligned.
int check_ints(const bea_tensor* t, int ndim) {
  if (t == nullptr) return BEA_ERR_ARG;
  if (t->ndim != ndim) return BEA_ERR_SHAPE;
  if (t->dtype != BEA_I32) return BEA_ERR_DTYPE;
  bool empty = false;
  for (int i = 0; i < ndim; ++i) {
    if (t->shape[i] < 0 || t->shape[i] > (int64_t(1) << 31) - 1) return BEA_ERR_SHAPE;
    if (t->stride[i] < 0) return BEA_ERR_ALIGN;
    empty = empty || t->shape[i] == 0;
  }
  if (empty) return BEA_OK;
  if (t->data == nullptr) return BEA_ERR_ARG;
  if (t->shape[ndim - 1] > 1 && t->stride[ndim - 1] != 1) return BEA_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(t->data) % 4 != 0) return BEA_ERR_ALIGN;
  return BEA_OK;
}

// A tensor that is written must not be broadcast: no stride 0 over several entries.
bool broadcast(const bea_tensor* t) {
  bool found = false;
  for (int i = 0; i < t->ndim; ++i) {
    if (t->shape[i] == 0) return false;
    found = found || (t->shape[i] > 1 && t->stride[i] == 0);
  }
  return found;
}

bool same_strides(const bea_tensor* a, const bea_tensor* b) {
  for (int i = 0; i < a->ndim; ++i)
    if (a->shape[i] > 1 && a->stride[i] != b->stride[i]) return false;
  return true;
}

// A [num_pages, page_size, h_kv, d] pair of caches.
int check_caches(const bea_tensor* k, const bea_tensor* v) {
  int rc;
  if ((rc = check_tensor(k, 4)) || (rc = check_tensor(v, 4))) return rc;
  if (k->dtype != v->dtype) return BEA_ERR_DTYPE;
  if (!same_shape(k, v)) return BEA_ERR_SHAPE;
  if (k->shape[1] < 1 || k->shape[0] * k->shape[1] > (int64_t(1) << 31) - 1) return BEA_ERR_SHAPE;
  return BEA_OK;
}

int check_paged_decode(const bea_tensor* q, const bea_tensor* k_cache, const bea_tensor* v_cache,
                       const bea_tensor* block_table, const bea_tensor* lens, const bea_tensor* out,
                       const bea_tensor* lse, float softmax_scale, int window_left, PagedDecodeParams* p) {
  int rc;
  if ((rc = check_tensor(q, 4)) || (rc = check_caches(k_cache, v_cache)) || (rc = check_ints(block_table, 2)) ||
      (rc = check_ints(lens, 1)) || (rc = check_tensor(out, 4)) || (rc = check_tensor(lse, 3)))
    return rc;
  if (q->dtype != k_cache->dtype || lse->dtype != BEA_F32) return BEA_ERR_DTYPE;
  if (out->dtype != q->dtype && out->dtype != BEA_F32) return BEA_ERR_DTYPE;
  const int64_t n = q->shape[0], h = q->shape[2], d = q->shape[3], hkv = k_cache->shape[2];
  if (q->shape[1] != 1 || !same_shape(out, q)) return BEA_ERR_SHAPE;
  if (lse->shape[0] != n || lse->shape[1] != h || lse->shape[2] != 1) return BEA_ERR_SHAPE;
  if (block_table->shape[0] != n || lens->shape[0] != n) return BEA_ERR_SHAPE;
  if (k_cache->shape[3] != d || hkv <= 0 || h % hkv != 0) return BEA_ERR_SHAPE;
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f) || window_left < -1) return BEA_ERR_ARG;
  if (broadcast(out) || broadcast(lse)) return BEA_ERR_ARG;
  if (q->dtype == BEA_BF16 ? (d != 64 && d != 128) : (d < 4 || d > 128 || d % 4 != 0)) return BEA_ERR_UNSUPPORTED;
  if (n * h > (int64_t(1) << 31) - 1 || h * d > (int64_t(1) << 31) - 1) return BEA_ERR_SHAPE;
  const int64_t page = k_cache->shape[1], max_pages = block_table->shape[1];
  const int64_t max_keys = max_pages * page;
  if (max_keys >= bea::kUnbounded) return BEA_ERR_SHAPE;
  if (!bea::paged_decode_fits(hkv, d, q->dtype == BEA_F32, max_keys)) return BEA_ERR_SHAPE;
  std::memset(p, 0, sizeof(*p));
  p->n = (int)n;
  p->h = (int)h;
  p->hkv = (int)hkv;
  p->d = (int)d;
  p->num_pages = (int)k_cache->shape[0];
  p->page = (int)page;
  p->page_shift = (page & (page - 1)) == 0 ? __builtin_ctzll((unsigned long long)page) : -1;
  p->max_pages = (int)max_pages;
  p->left = window_left < 0 || window_left > bea::kUnbounded ? bea::kUnbounded : window_left;
  p->is_f32 = q->dtype == BEA_F32;
  p->out_is_f32 = out->dtype == BEA_F32;
  p->scale = softmax_scale;
  p->q = seq4(q);
  p->out = seq4(out);
  p->kc = seq4(k_cache);
  p->vc = seq4(v_cache);
  p->lse = lse3(lse);
  p->table = static_cast<const int32_t*>(block_table->data);
  p->table_stride = block_table->stride[0];
  p->lens = static_cast<const int32_t*>(lens->data);
  return BEA_OK;
}

// One of rope's (input, output) pairs.
int check_rope_pair(const bea_tensor* x, const bea_tensor* y, const bea_tensor* like) {
  int rc;
  if ((rc = check_tensor(x, 4)) || (rc = check_tensor(y, 4))) return rc;
  if (x->dtype != like->dtype || y->dtype != like->dtype) return BEA_ERR_DTYPE;
  if (!same_shape(x, y)) return BEA_ERR_SHAPE;
  if (x->shape[0] != like->shape[0] || x->shape[1] != like->shape[1] || x->shape[3] != like->shape[3])
    return BEA_ERR_SHAPE;
  if (broadcast(y)) return BEA_ERR_ARG;
  if (x->data == y->data && !same_strides(x, y)) return BEA_ERR_ARG;
  return BEA_OK;
}

uint64_t fraction_of_turn(double freq) {
  // Rounded; of a negative one's size, which loses no bits where it is small. It is at most 1 - 2^-53, so its product is
  // below 2^64.
  const double turns = std::fabs(freq) * 0.15915494309189533577;  // 1 / (2 pi)
  const uint64_t step = static_cast<uint64_t>(std::nearbyint((turns - std::floor(turns)) * 0x1p64));
  return freq < 0 ? 0 - step : step;
}

}  // namespace abi
}  // namespace bea

using namespace bea::abi;

namespace {

const int32_t* ints(const bea_tensor* t) { return static_cast<const int32_t*>(t->data); }
int32_t* ints_out(const bea_tensor* t) { return static_cast<int32_t*>(t->data); }

}  // namespace

extern "C" {

int bea_rope_axes(const bea_tensor* q, const bea_tensor* k, const bea_tensor* positions, const int32_t* axis_of_pair,
                  const double* freq, int inverse, const bea_tensor* q_out, const bea_tensor* k_out, void* stream) {
  int rc;
  if (q == nullptr || q_out == nullptr || axis_of_pair == nullptr || freq == nullptr) return BEA_ERR_ARG;
  if ((k == nullptr) != (k_out == nullptr)) return BEA_ERR_ARG;
  if (inverse != 0 && inverse != 1) return BEA_ERR_ARG;
  if ((rc = check_tensor(q, 4)) || (rc = check_rope_pair(q, q_out, q))) return rc;
  if (k != nullptr && (rc = check_rope_pair(k, k_out, q))) return rc;
  if ((rc = check_ints(positions, 3))) return rc;
  const int64_t axes = positions->shape[0], d = q->shape[3];
  if (axes < 1 || axes > bea::kRopeMaxAxes) return BEA_ERR_SHAPE;
  if (positions->shape[1] != q->shape[0] || positions->shape[2] != q->shape[1]) return BEA_ERR_SHAPE;
  if (d < 1 || d > 2 * bea::kRopeMaxPairs || d % (q->dtype == BEA_F32 ? 8 : 16) != 0) return BEA_ERR_UNSUPPORTED;
  const int64_t hk = k != nullptr ? k->shape[2] : 0;
  if (q->shape[2] + hk > (int64_t(1) << 30)) return BEA_ERR_SHAPE;
  bea::RopeParams p;
  std::memset(&p, 0, sizeof(p));
  for (int i = 0; i < d / 2; ++i) {
    if (axis_of_pair[i] < 0 || axis_of_pair[i] >= axes || !std::isfinite(freq[i])) return BEA_ERR_ARG;
    p.turn[i] = fraction_of_turn(freq[i]);
    p.axis[i] = static_cast<uint8_t>(axis_of_pair[i]);
  }
  p.n = (int)q->shape[0];
  p.l = (int)q->shape[1];
  p.hq = (int)q->shape[2];
  p.hk = (int)hk;
  p.d = (int)d;
  p.is_f32 = q->dtype == BEA_F32;
  p.inverse = inverse;
  p.q = seq4(q);
  p.qo = seq4(q_out);
  if (k != nullptr) {
    p.k = seq4(k);
    p.ko = seq4(k_out);
  }
  p.pos = ints(positions);
  p.pos_sa = positions->stride[0];
  p.pos_sn = positions->stride[1];
  int launches = 0;
  if (p.n == 0 || p.l == 0 || p.hq + p.hk == 0) return finish(cudaSuccess, 0);
  return finish(bea::launch_rope(p, static_cast<cudaStream_t>(stream), &launches), launches);
}

int bea_paged_plan(const bea_tensor* lens, const bea_tensor* new_lens, const bea_tensor* block_table,
                   const bea_tensor* free_pages, const bea_tensor* n_free, int64_t page_size,
                   const bea_tensor* slot_map, const bea_tensor* positions, const bea_tensor* cu_new,
                   const bea_tensor* cu_pages, const bea_tensor* lens_out, const bea_tensor* n_free_out,
                   void* stream) {
  int rc;
  for (const bea_tensor* t : {lens, new_lens, free_pages, n_free, slot_map, positions, cu_new, cu_pages, lens_out,
                              n_free_out})
    if ((rc = check_ints(t, 1))) return rc;
  if ((rc = check_ints(block_table, 2))) return rc;
  const int64_t n = lens->shape[0];
  if (new_lens->shape[0] != n || block_table->shape[0] != n || lens_out->shape[0] != n) return BEA_ERR_SHAPE;
  if (cu_new->shape[0] != n + 1 || cu_pages->shape[0] != n + 1) return BEA_ERR_SHAPE;
  if (n_free->shape[0] != 1 || n_free_out->shape[0] != 1) return BEA_ERR_SHAPE;
  if (slot_map->shape[0] != positions->shape[0]) return BEA_ERR_SHAPE;
  if (page_size < 1 || page_size > (int64_t(1) << 20)) return BEA_ERR_ARG;
  if (block_table->shape[1] * page_size >= bea::kUnbounded) return BEA_ERR_SHAPE;
  if (n > 1 && block_table->stride[0] < block_table->shape[1]) return BEA_ERR_ARG;
  bea::PlanParams p;
  std::memset(&p, 0, sizeof(p));
  p.n = (int)n;
  p.max_pages = (int)block_table->shape[1];
  p.capacity = (int)slot_map->shape[0];
  p.n_pool = (int)free_pages->shape[0];
  p.page = (int)page_size;
  p.lens = ints(lens);
  p.new_lens = ints(new_lens);
  p.n_free = ints(n_free);
  p.table = ints_out(block_table);
  p.table_stride = block_table->stride[0];
  p.pool = ints_out(free_pages);
  p.slot_map = ints_out(slot_map);
  p.positions = ints_out(positions);
  p.cu_new = ints_out(cu_new);
  p.cu_pages = ints_out(cu_pages);
  p.lens_out = ints_out(lens_out);
  p.n_free_out = ints_out(n_free_out);
  if ((rc = status_ptr_for_current_device(&p.status))) return rc;
  int launches = 0;
  return finish(bea::launch_paged_plan(p, static_cast<cudaStream_t>(stream), &launches), launches);
}

int bea_paged_write(const bea_tensor* k, const bea_tensor* v, const bea_tensor* slot_map, const bea_tensor* k_cache,
                    const bea_tensor* v_cache, void* stream) {
  int rc;
  if ((rc = check_tensor(k, 4)) || (rc = check_tensor(v, 4)) || (rc = check_ints(slot_map, 1)) ||
      (rc = check_caches(k_cache, v_cache)))
    return rc;
  if (k->dtype != v->dtype || k->dtype != k_cache->dtype) return BEA_ERR_DTYPE;
  if (!same_shape(k, v)) return BEA_ERR_SHAPE;
  if (k->shape[2] != k_cache->shape[2] || k->shape[3] != k_cache->shape[3]) return BEA_ERR_SHAPE;
  if (k->shape[0] * k->shape[1] > (int64_t(1) << 31) - 1 || slot_map->shape[0] != k->shape[0] * k->shape[1])
    return BEA_ERR_SHAPE;
  if (broadcast(k_cache) || broadcast(v_cache)) return BEA_ERR_ARG;
  const int es = k->dtype == BEA_F32 ? 4 : 2;
  if (k->shape[3] * es % 16 != 0) return BEA_ERR_UNSUPPORTED;
  if (k->shape[2] * (k->shape[3] * es / 16) > (int64_t(1) << 31) - 1) return BEA_ERR_SHAPE;
  bea::PagedWriteParams p;
  std::memset(&p, 0, sizeof(p));
  p.n = (int)k->shape[0];
  p.l = (int)k->shape[1];
  p.hkv = (int)k->shape[2];
  p.row_vecs = (int)(k->shape[3] * es / 16);
  p.es = es;
  p.num_slots = (int)(k_cache->shape[0] * k_cache->shape[1]);
  p.page = (int)k_cache->shape[1];
  p.k = seq4(k);
  p.v = seq4(v);
  p.k_cache = seq4(k_cache);
  p.v_cache = seq4(v_cache);
  p.slot_map = ints(slot_map);
  if (p.n == 0 || p.l == 0 || p.hkv == 0 || p.row_vecs == 0) return finish(cudaSuccess, 0);
  if ((rc = status_ptr_for_current_device(&p.status))) return rc;
  int launches = 0;
  return finish(bea::launch_paged_write(p, static_cast<cudaStream_t>(stream), &launches), launches);
}

size_t bea_paged_decode_workspace_size(int64_t h, int64_t h_kv, int64_t d, int64_t max_keys) {
  if (h < 0 || h_kv <= 0 || d < 0 || max_keys < 0) return 0;
  return bea::paged_decode_workspace(h, h_kv, d, max_keys);
}

int bea_paged_decode(const bea_tensor* q, const bea_tensor* k_cache, const bea_tensor* v_cache,
                     const bea_tensor* block_table, const bea_tensor* lens, const bea_tensor* out,
                     const bea_tensor* lse, float softmax_scale, int window_left, void* workspace,
                     size_t workspace_bytes, void* stream) {
  bea::PagedDecodeParams p;
  int rc = check_paged_decode(q, k_cache, v_cache, block_table, lens, out, lse, softmax_scale, window_left, &p);
  if (rc) return rc;
  const size_t need = bea::paged_decode_workspace(p.h, p.hkv, p.d, (int64_t)p.max_pages * p.page);
  if (need > 0 && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || workspace_bytes < need))
    return BEA_ERR_WORKSPACE;
  p.ws = workspace;
  if (p.n == 0 || p.h == 0) return finish(cudaSuccess, 0);
  if ((rc = status_ptr_for_current_device(&p.status))) return rc;
  int launches = 0;
  return finish(bea::launch_paged_decode(p, static_cast<cudaStream_t>(stream), &launches), launches);
}

}  // extern "C"
