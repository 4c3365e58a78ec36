// C entry points of the normed and laid-out rotary calls: argument checks (all
// before any CUDA call) and dispatch.
#include <cmath>
#include <cstring>

#include "../../include/bea.h"
#include "abi_internal.h"
#include "norm_rope.cuh"

using namespace bea::abi;

namespace {

int check_weight(const bea_tensor* w, int64_t d) {
  if (w == nullptr) return BEA_OK;
  int rc;
  if ((rc = check_tensor(w, 1))) return rc;
  return w->shape[0] == d ? BEA_OK : BEA_ERR_SHAPE;
}
int check_weight_grad(const bea_tensor* g, const bea_tensor* w, int64_t d) {
  if (g == nullptr) return BEA_OK;
  if (w == nullptr) return BEA_ERR_ARG;
  int rc;
  if ((rc = check_weight(g, d))) return rc;
  return g->dtype == w->dtype ? BEA_OK : BEA_ERR_DTYPE;
}

// What the forward and the gradient have in common. q_out, k_out: what is written, of x's shape.
int check_norm_rope(const bea_tensor* q, const bea_tensor* k, const bea_tensor* positions, const int32_t* axis_of_pair,
                    const double* freq, int pairs, int interleaved, float amplitude, const bea_tensor* q_weight,
                    const bea_tensor* k_weight, int norm, float eps, const bea_tensor* q_out, const bea_tensor* k_out,
                    bea::NormRopeParams* p) {
  int rc;
  if (q == nullptr || q_out == nullptr) return BEA_ERR_ARG;
  if ((k == nullptr) != (k_out == nullptr) || (k == nullptr && k_weight != nullptr)) return BEA_ERR_ARG;
  if ((interleaved != 0 && interleaved != 1) || (norm != 0 && norm != 1)) return BEA_ERR_ARG;
  if (!std::isfinite(amplitude) || !std::isfinite(eps) || eps < 0.f) return BEA_ERR_ARG;
  if (norm == 0 && (q_weight != nullptr || k_weight != nullptr)) return BEA_ERR_ARG;
  if ((rc = check_tensor(q, 4)) || (rc = check_rope_pair(q, q_out, q))) return rc;
  if (k != nullptr && (rc = check_rope_pair(k, k_out, q))) return rc;
  if ((rc = check_ints(positions, 3))) return rc;
  const int64_t axes = positions->shape[0], d = q->shape[3];
  if (axes < 1 || axes > bea::kRopeMaxAxes) return BEA_ERR_SHAPE;
  if (positions->shape[1] != q->shape[0] || positions->shape[2] != q->shape[1]) return BEA_ERR_SHAPE;
  const int piece = q->dtype == BEA_F32 ? 4 : 8;
  if (d < 1 || d > 2 * bea::kRopeMaxPairs || d % (2 * piece) != 0) return BEA_ERR_UNSUPPORTED;
  if (pairs < 0 || 2 * (int64_t)pairs > d) return BEA_ERR_ARG;
  if (!interleaved && pairs % piece != 0) return BEA_ERR_UNSUPPORTED;
  if (pairs > 0 && (axis_of_pair == nullptr || freq == nullptr)) return BEA_ERR_ARG;
  const int64_t hk = k != nullptr ? k->shape[2] : 0;
  if (q->shape[2] + hk > (int64_t(1) << 30)) return BEA_ERR_SHAPE;
  if ((rc = check_weight(q_weight, d)) || (rc = check_weight(k_weight, d))) return rc;
  std::memset(p, 0, sizeof(*p));
  for (int i = 0; i < pairs; ++i) {
    if (axis_of_pair[i] < 0 || axis_of_pair[i] >= axes || !std::isfinite(freq[i])) return BEA_ERR_ARG;
    p->turn[i] = fraction_of_turn(freq[i]);
    p->axis[i] = static_cast<uint8_t>(axis_of_pair[i]);
  }
  p->n = (int)q->shape[0];
  p->l = (int)q->shape[1];
  p->hq = (int)q->shape[2];
  p->hk = (int)hk;
  p->d = (int)d;
  p->pairs = pairs;
  p->is_f32 = q->dtype == BEA_F32;
  p->interleaved = interleaved;
  p->norm = norm;
  p->eps = eps;
  p->amplitude = amplitude;
  p->q = seq4(q);
  p->qo = seq4(q_out);
  if (k != nullptr) {
    p->k = seq4(k);
    p->ko = seq4(k_out);
  }
  if (q_weight != nullptr) p->wq = q_weight->data, p->wq_f32 = q_weight->dtype == BEA_F32;
  if (k_weight != nullptr) p->wk = k_weight->data, p->wk_f32 = k_weight->dtype == BEA_F32;
  p->pos = static_cast<const int32_t*>(positions->data);
  p->pos_sa = positions->stride[0];
  p->pos_sn = positions->stride[1];
  return BEA_OK;
}

}  // namespace

extern "C" {

int bea_norm_rope_axes(const bea_tensor* q, const bea_tensor* k, const bea_tensor* positions,
                       const int32_t* axis_of_pair, const double* freq, int pairs, int interleaved, float amplitude,
                       int inverse, const bea_tensor* q_weight, const bea_tensor* k_weight, int norm, float eps,
                       const bea_tensor* q_out, const bea_tensor* k_out, void* stream) {
  bea::NormRopeParams p;
  const int rc = check_norm_rope(q, k, positions, axis_of_pair, freq, pairs, interleaved, amplitude, q_weight, k_weight,
                                 norm, eps, q_out, k_out, &p);
  if (rc) return rc;
  if ((inverse != 0 && inverse != 1) || (norm == 1 && inverse == 1)) return BEA_ERR_ARG;
  p.inverse = inverse;
  int launches = 0;
  if (p.n == 0 || p.l == 0 || p.hq + p.hk == 0) return finish(cudaSuccess, 0);
  return finish(bea::launch_norm_rope(p, static_cast<cudaStream_t>(stream), &launches), launches);
}

size_t bea_norm_rope_axes_bwd_workspace_size(int64_t d) { return d <= 0 ? 0 : bea::norm_rope_bwd_workspace(d); }

int bea_norm_rope_axes_bwd(const bea_tensor* q, const bea_tensor* k, const bea_tensor* dq_out, const bea_tensor* dk_out,
                           const bea_tensor* positions, const int32_t* axis_of_pair, const double* freq, int pairs,
                           int interleaved, float amplitude, const bea_tensor* q_weight, const bea_tensor* k_weight,
                           float eps, const bea_tensor* dq, const bea_tensor* dk, const bea_tensor* dq_weight,
                           const bea_tensor* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
  bea::NormRopeParams p;
  int rc = check_norm_rope(q, k, positions, axis_of_pair, freq, pairs, interleaved, amplitude, q_weight, k_weight, 1, eps,
                           dq, dk, &p);
  if (rc) return rc;
  if (dq_out == nullptr || (k == nullptr) != (dk_out == nullptr)) return BEA_ERR_ARG;
  if ((rc = check_tensor(dq_out, 4)) || (k != nullptr && (rc = check_tensor(dk_out, 4)))) return rc;
  if (dq_out->dtype != q->dtype || (k != nullptr && dk_out->dtype != q->dtype)) return BEA_ERR_DTYPE;
  if (!same_shape(dq_out, q) || (k != nullptr && !same_shape(dk_out, k))) return BEA_ERR_SHAPE;
  const int64_t d = q->shape[3];
  if ((rc = check_weight_grad(dq_weight, q_weight, d)) || (rc = check_weight_grad(dk_weight, k_weight, d))) return rc;
  const bool sums = dq_weight != nullptr || dk_weight != nullptr;
  if (sums && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 256 != 0 ||
               workspace_bytes < bea::norm_rope_bwd_workspace(d)))
    return BEA_ERR_WORKSPACE;
  p.gq = seq4(dq_out);
  if (k != nullptr) p.gk = seq4(dk_out);
  p.partial = static_cast<float*>(workspace);
  if (dq_weight != nullptr) p.dwq = dq_weight->data;
  if (dk_weight != nullptr) p.dwk = dk_weight->data;
  int launches = 0;
  return finish(bea::launch_norm_rope_bwd(p, static_cast<cudaStream_t>(stream), &launches), launches);
}

}  // extern "C"
