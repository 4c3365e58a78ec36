// C entry point of attention over a shared prefix: argument checks (all before
// any CUDA call) and dispatch.
#include <cstring>

#include "../../include/bea.h"
#include "abi_internal.h"
#include "paged_shared.cuh"

using namespace bea::abi;

extern "C" {

size_t bea_paged_decode_shared_workspace_size(int64_t n, int64_t h, int64_t h_kv, int64_t d, int64_t max_keys,
                                              int64_t groups) {
  if (n < 0 || h < 0 || h_kv <= 0 || d < 0 || max_keys < 0 || groups < 0) return 0;
  // what bea_paged_decode_shared refuses anyway, and products past 64 bits
  constexpr int64_t most = int64_t(1) << 31;
  if (n > most || h > most || n * h > most || d < 1 || d > 128 || max_keys > bea::kUnbounded || groups > bea::kMaxGroups) return 0;
  return bea::paged_shared_workspace(n, h, h_kv, d, max_keys, groups);
}

int bea_paged_decode_shared(const bea_tensor* q, const bea_tensor* k_cache, const bea_tensor* v_cache,
                            const bea_tensor* block_table, const bea_tensor* lens, const bea_tensor* group_rows,
                            const bea_tensor* shared_lens, const bea_tensor* out, const bea_tensor* lse,
                            float softmax_scale, void* workspace, size_t workspace_bytes, void* stream) {
  bea::PagedSharedParams p;
  std::memset(&p, 0, sizeof(p));
  int rc = check_paged_decode(q, k_cache, v_cache, block_table, lens, out, lse, softmax_scale, -1, &p.d);
  if (rc) return rc;
  if ((rc = check_ints(group_rows, 1)) || (rc = check_ints(shared_lens, 1))) return rc;
  if (q->dtype != BEA_BF16) return BEA_ERR_UNSUPPORTED;
  const int64_t groups = shared_lens->shape[0], max_keys = (int64_t)p.d.max_pages * p.d.page;
  if (group_rows->shape[0] != groups + 1) return BEA_ERR_SHAPE;
  if (groups > bea::kMaxGroups) return BEA_ERR_UNSUPPORTED;
  if (!bea::paged_shared_fits(p.d.n, p.d.h, p.d.hkv, max_keys, groups)) return BEA_ERR_SHAPE;
  const size_t need = bea::paged_shared_workspace(p.d.n, p.d.h, p.d.hkv, p.d.d, max_keys, groups);
  if (need > 0 && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 || workspace_bytes < need))
    return BEA_ERR_WORKSPACE;
  p.d.ws = workspace;
  p.groups = (int)groups;
  p.group_rows = static_cast<const int32_t*>(group_rows->data);
  p.shared_lens = static_cast<const int32_t*>(shared_lens->data);
  if (p.d.n == 0 || p.d.h == 0) return finish(cudaSuccess, 0);
  if ((rc = status_ptr_for_current_device(&p.d.status))) return rc;
  int launches = 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // (no copies by box from a cache whose pages, tokens or heads lie on one another)
  if (bea::paged_shared_is_plain(p.d, groups) || broadcast(k_cache) || broadcast(v_cache))
    return finish(bea::launch_paged_decode(p.d, s, &launches), launches);
  bea::PageMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  int box = bea::paged_shared_box(p.d.page);
  for (int i = 0; i < bea::kPageMaps && box <= 128 && box <= p.d.page; ++i, box *= 2)
    if ((rc = make_page_map(k_cache, box, &maps.k[i])) || (rc = make_page_map(v_cache, box, &maps.v[i]))) return rc;
  return finish(bea::launch_paged_shared(p, maps, s, &launches), launches);
}

}  // extern "C"
