// C ABI of routing from scores (declared in include/qmoe.h): contract checks
// and enqueue.
#include <hip/hip_runtime.h>

#include <cmath>

#include "kernels/route_scored.h"
#include "qmoe_checks.h"

using namespace qmoe;

namespace {

constexpr int64_t kMaxRoute = 1024;              // experts of a router row: 16 a lane
constexpr int64_t kMaxSlots = int64_t(1) << 30;  // T k

qmoe_status check_scored(const qmoe_tensor* logits, const qmoe_route_attrs* a, int64_t k, RouteScored* r) {
  if (logits->rank != 2) return QMOE_ERR_SHAPE;
  if (logits->dtype != QMOE_F32) return QMOE_ERR_DTYPE;
  const int64_t T = logits->dims[0], E = logits->dims[1];
  if (T < 0 || E < 0) return QMOE_ERR_SHAPE;
  if (a->scores != QMOE_SCORES_SOFTMAX && a->scores != QMOE_SCORES_SIGMOID) return QMOE_ERR_ATTR;
  if (a->normalize_routing_weights != 0 && a->normalize_routing_weights != 1) return QMOE_ERR_ATTR;
  if (a->group_top != 1 && a->group_top != 2) return QMOE_ERR_ATTR;
  if (!std::isfinite(a->scale)) return QMOE_ERR_ATTR;
  if (a->groups < 1 || E % a->groups != 0 || a->kept_groups < 1 || a->kept_groups > a->groups) return QMOE_ERR_ATTR;
  if (k < 1 || k > E / a->groups * a->kept_groups) return QMOE_ERR_ATTR;
  if (E > kMaxRoute || a->groups > kMaxRouteGroups || T >= kMaxSlots || T * k >= kMaxSlots) return QMOE_ERR_UNSUPPORTED;
  *r = {(int)E, (int)k, a->scores == QMOE_SCORES_SIGMOID, a->groups, a->kept_groups, a->group_top,
        a->normalize_routing_weights, a->scale};
  return QMOE_OK;
}

}  // namespace

extern "C" {

void qmoe_route_attrs_default(qmoe_route_attrs* a) { *a = {1, QMOE_SCORES_SOFTMAX, 1, 1, 2, 0, 1.f}; }

qmoe_status qmoe_route_scored(const qmoe_tensor* router_probs, const qmoe_tensor* bias, const qmoe_route_attrs* attrs,
                              const qmoe_tensor* indices, const qmoe_tensor* weights, void* stream) {
  if (!router_probs || !attrs || !indices || !weights) return QMOE_ERR_NULL;
  RouteScored r;
  qmoe_status st = check_scored(router_probs, attrs, attrs->k, &r);
  if (st != QMOE_OK) return st;
  const int64_t T = router_probs->dims[0], k = attrs->k;
  if (indices->dtype != QMOE_I32 || weights->dtype != QMOE_F32 || (bias && bias->dtype != QMOE_F32)) return QMOE_ERR_DTYPE;
  if (!is(indices, {T, k}) || !is(weights, {T, k}) || (bias && !is(bias, {r.E}))) return QMOE_ERR_SHAPE;
  if (T == 0) return QMOE_OK;
  st = check_data({router_probs, bias, indices, weights});
  if (st != QMOE_OK) return st;
  return launch_route_scored(static_cast<const float*>(router_probs->data), static_cast<const float*>(data_of(bias)),
                             (int)T, r, static_cast<int*>(data_of(indices)), static_cast<float*>(data_of(weights)),
                             reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? QMOE_OK
             : QMOE_ERR_HIP;
}

qmoe_status qmoe_route_scored_backward(const qmoe_tensor* grad_weights, const qmoe_tensor* router_probs,
                                       const qmoe_tensor* indices, const qmoe_route_attrs* attrs,
                                       const qmoe_tensor* grad_router_probs, void* stream) {
  if (!grad_weights || !router_probs || !indices || !attrs || !grad_router_probs) return QMOE_ERR_NULL;
  if (indices->rank != 2) return QMOE_ERR_SHAPE;
  RouteScored r;
  const int64_t k = indices->dims[1];
  qmoe_status st = check_scored(router_probs, attrs, k, &r);
  if (st != QMOE_OK) return st;
  const int64_t T = router_probs->dims[0];
  if (!index_code(indices->dtype) || grad_weights->dtype != QMOE_F32 || grad_router_probs->dtype != QMOE_F32)
    return QMOE_ERR_DTYPE;
  if (!is(indices, {T, k}) || !is(grad_weights, {T, k}) || !is(grad_router_probs, {T, r.E})) return QMOE_ERR_SHAPE;
  if (T == 0) return QMOE_OK;
  st = check_data({grad_weights, router_probs, indices, grad_router_probs});
  if (st != QMOE_OK) return st;
  return launch_route_scored_grad(static_cast<const float*>(grad_weights->data),
                                  static_cast<const float*>(router_probs->data), indices->data,
                                  indices->dtype == QMOE_I64, (int)T, r,
                                  static_cast<float*>(data_of(grad_router_probs)),
                                  reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? QMOE_OK
             : QMOE_ERR_HIP;
}

}  // extern "C"
