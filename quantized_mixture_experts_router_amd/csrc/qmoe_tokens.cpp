// C ABI of routing weights, token dispatch and combine with their gradients
// (declared in include/qmoe.h): contract checks and enqueue.
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "kernels/tokens.h"
#include "qmoe.h"

using namespace qmoe;

namespace {

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxRoute = 1024;               // experts of a router row: 16 a lane
constexpr int64_t kMaxSort = 1023;                // experts sorted by (one more bucket for dropped slots)
constexpr int64_t kMaxSlots = int64_t(1) << 30;   // T k

int64_t numel(const qmoe_tensor* t) {
  int64_t n = 1;
  for (int i = 0; i < t->rank; ++i) n *= t->dims[i];
  return n;
}

bool is(const qmoe_tensor* t, std::initializer_list<int64_t> dims) {
  if (t->rank != (int)dims.size()) return false;
  int i = 0;
  for (int64_t d : dims)
    if (t->dims[i++] != d) return false;
  return true;
}

bool float_code(int32_t dt) { return dt == QMOE_F32 || dt == QMOE_F16 || dt == QMOE_BF16; }
bool index_code(int32_t dt) { return dt == QMOE_I32 || dt == QMOE_I64; }
int row_type(int32_t dt) { return dt == QMOE_F32 ? ROW_F32 : dt == QMOE_F16 ? ROW_F16 : ROW_BF16; }
uintptr_t esize(int32_t dt) { return dt == QMOE_I64 ? 8 : dt == QMOE_F16 || dt == QMOE_BF16 ? 2 : 4; }

// Pointers present where there are elements, aligned to the element.
qmoe_status check_data(std::initializer_list<const qmoe_tensor*> ts) {
  for (const qmoe_tensor* t : ts) {
    if (!t) continue;
    if (numel(t) > 0 && !t->data) return QMOE_ERR_NULL;
    if (!aligned_to(t->data, esize(t->dtype))) return QMOE_ERR_ALIGN;
  }
  return QMOE_OK;
}

qmoe_status check_route(const qmoe_tensor* logits, int64_t k, int32_t routing, int32_t normalize) {
  if (logits->rank != 2) return QMOE_ERR_SHAPE;
  if (logits->dtype != QMOE_F32) return QMOE_ERR_DTYPE;
  if (logits->dims[0] < 0 || logits->dims[1] < 0) return QMOE_ERR_SHAPE;
  if (routing != QMOE_ROUTE_QMOE && routing != QMOE_ROUTE_MOE) return QMOE_ERR_ATTR;
  if (normalize != 0 && normalize != 1) return QMOE_ERR_ATTR;
  if (k < 1 || k > logits->dims[1]) return QMOE_ERR_ATTR;
  if (logits->dims[1] > kMaxRoute || logits->dims[0] >= kMaxSlots || logits->dims[0] * k >= kMaxSlots)
    return QMOE_ERR_UNSUPPORTED;
  return QMOE_OK;
}

bool over_all(int32_t routing, int32_t normalize) { return routing == QMOE_ROUTE_MOE && !normalize; }

// inverse [T, k], rows [T k, H] and tokens [T, H] of one type; any may be
// NULL but inverse.
qmoe_status check_rows(const qmoe_tensor* inverse, std::initializer_list<const qmoe_tensor*> rows,
                       std::initializer_list<const qmoe_tensor*> tokens) {
  if (inverse->rank != 2) return QMOE_ERR_SHAPE;
  const qmoe_tensor* first = nullptr;
  for (const qmoe_tensor* t : rows) {
    if (!t) continue;
    if (!first) first = t;
    if (t->rank != 2) return QMOE_ERR_SHAPE;
  }
  for (const qmoe_tensor* t : tokens) {
    if (!t) continue;
    if (!first) first = t;
    if (t->rank != 2) return QMOE_ERR_SHAPE;
  }
  if (inverse->dtype != QMOE_I32) return QMOE_ERR_DTYPE;
  if (!float_code(first->dtype)) return QMOE_ERR_DTYPE;
  for (const qmoe_tensor* t : rows)
    if (t && t->dtype != first->dtype) return QMOE_ERR_DTYPE;
  for (const qmoe_tensor* t : tokens)
    if (t && t->dtype != first->dtype) return QMOE_ERR_DTYPE;
  const int64_t T = inverse->dims[0], k = inverse->dims[1], H = first->dims[1];
  if (T < 0 || k < 0 || H < 0) return QMOE_ERR_SHAPE;
  if (T >= kMaxSlots || k >= kMaxSlots || T * k >= kMaxSlots || H >= kMaxSlots) return QMOE_ERR_UNSUPPORTED;
  for (const qmoe_tensor* t : rows)
    if (t && !is(t, {T * k, H})) return QMOE_ERR_SHAPE;
  for (const qmoe_tensor* t : tokens)
    if (t && !is(t, {T, H})) return QMOE_ERR_SHAPE;
  return QMOE_OK;
}

// At most 65535 blocks of 256 pieces a row.
bool row_too_long(int64_t H) { return H > int64_t(65535) * 256; }

}  // namespace

extern "C" {

qmoe_status qmoe_route(const qmoe_tensor* router_probs, int32_t k, int32_t routing,
                       int32_t normalize_routing_weights, const qmoe_tensor* indices, const qmoe_tensor* weights,
                       void* stream) {
  if (!router_probs || !indices || !weights) return QMOE_ERR_NULL;
  qmoe_status st = check_route(router_probs, k, routing, normalize_routing_weights);
  if (st != QMOE_OK) return st;
  const int64_t T = router_probs->dims[0], E = router_probs->dims[1];
  if (indices->dtype != QMOE_I32 || weights->dtype != QMOE_F32) return QMOE_ERR_DTYPE;
  if (!is(indices, {T, k}) || !is(weights, {T, k})) return QMOE_ERR_SHAPE;
  if (T == 0) return QMOE_OK;
  st = check_data({router_probs, indices, weights});
  if (st != QMOE_OK) return st;
  return launch_route_topk(static_cast<const float*>(router_probs->data), (int)T, (int)E, k,
                           over_all(routing, normalize_routing_weights),
                           static_cast<int*>(const_cast<void*>(indices->data)),
                           static_cast<float*>(const_cast<void*>(weights->data)),
                           reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? QMOE_OK
             : QMOE_ERR_HIP;
}

qmoe_status qmoe_route_backward(const qmoe_tensor* grad_weights, const qmoe_tensor* router_probs,
                                const qmoe_tensor* indices, int32_t routing, int32_t normalize_routing_weights,
                                const qmoe_tensor* grad_router_probs, void* stream) {
  if (!grad_weights || !router_probs || !indices || !grad_router_probs) return QMOE_ERR_NULL;
  if (indices->rank != 2) return QMOE_ERR_SHAPE;
  const int64_t k = indices->dims[1];
  if (k < 0 || k > kMaxRoute) return QMOE_ERR_ATTR;
  qmoe_status st = check_route(router_probs, k, routing, normalize_routing_weights);
  if (st != QMOE_OK) return st;
  const int64_t T = router_probs->dims[0], E = router_probs->dims[1];
  if (!index_code(indices->dtype) || grad_weights->dtype != QMOE_F32 || grad_router_probs->dtype != QMOE_F32)
    return QMOE_ERR_DTYPE;
  if (!is(indices, {T, k}) || !is(grad_weights, {T, k}) || !is(grad_router_probs, {T, E})) return QMOE_ERR_SHAPE;
  if (T == 0) return QMOE_OK;
  st = check_data({grad_weights, router_probs, indices, grad_router_probs});
  if (st != QMOE_OK) return st;
  return launch_route_grad(static_cast<const float*>(grad_weights->data),
                           static_cast<const float*>(router_probs->data), indices->data, indices->dtype == QMOE_I64,
                           (int)T, (int)E, (int)k, over_all(routing, normalize_routing_weights),
                           static_cast<float*>(const_cast<void*>(grad_router_probs->data)),
                           reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? QMOE_OK
             : QMOE_ERR_HIP;
}

}  // extern "C"

namespace {

qmoe_status check_dispatch(const qmoe_tensor* input, const qmoe_tensor* indices, int64_t experts,
                           const qmoe_tensor* rows, const qmoe_tensor* offsets, const qmoe_tensor* perm,
                           const qmoe_tensor* inverse, size_t* bytes) {
  if (!input || !indices) return QMOE_ERR_NULL;
  if (input->rank != 2 || indices->rank != 2) return QMOE_ERR_SHAPE;
  if (!float_code(input->dtype) || !index_code(indices->dtype)) return QMOE_ERR_DTYPE;
  if (experts < 0) return QMOE_ERR_ATTR;
  const int64_t T = indices->dims[0], k = indices->dims[1];
  if (T < 0 || k < 0 || input->dims[1] < 0 || input->dims[0] != T) return QMOE_ERR_SHAPE;
  if (experts > kMaxSort || T >= kMaxSlots || k >= kMaxSlots || T * k >= kMaxSlots || row_too_long(input->dims[1]))
    return QMOE_ERR_UNSUPPORTED;
  if (rows && rows->dtype != input->dtype) return QMOE_ERR_DTYPE;
  for (const qmoe_tensor* t : {offsets, perm, inverse})
    if (t && t->dtype != QMOE_I32) return QMOE_ERR_DTYPE;
  if (rows && !is(rows, {T * k, input->dims[1]})) return QMOE_ERR_SHAPE;
  if (offsets && !is(offsets, {experts + 1})) return QMOE_ERR_SHAPE;
  if (perm && !is(perm, {T * k})) return QMOE_ERR_SHAPE;
  if (inverse && !is(inverse, {T, k})) return QMOE_ERR_SHAPE;
  const int64_t S = T * k, chunk = sort_chunk(S), n = (S + chunk - 1) / chunk;
  *bytes = S > kSortSelf ? (size_t)(n * (experts + 1)) * sizeof(int32_t) : 0;
  return QMOE_OK;
}

}  // namespace

extern "C" {

qmoe_status qmoe_dispatch_workspace_size(const qmoe_tensor* input, const qmoe_tensor* indices, int64_t experts,
                                         size_t* bytes) {
  if (!bytes) return QMOE_ERR_NULL;
  return check_dispatch(input, indices, experts, nullptr, nullptr, nullptr, nullptr, bytes);
}

qmoe_status qmoe_dispatch(const qmoe_tensor* input, const qmoe_tensor* indices, int64_t experts,
                          const qmoe_tensor* rows, const qmoe_tensor* offsets, const qmoe_tensor* perm,
                          const qmoe_tensor* inverse, void* workspace, size_t workspace_bytes, void* stream) {
  if (!rows || !offsets || !inverse) return QMOE_ERR_NULL;
  size_t need = 0;
  qmoe_status st = check_dispatch(input, indices, experts, rows, offsets, perm, inverse, &need);
  if (st != QMOE_OK) return st;
  st = check_data({input, indices, rows, offsets, perm, inverse});
  if (st != QMOE_OK) return st;
  if (need > 0) {
    if (!workspace) return QMOE_ERR_NULL;
    if (workspace_bytes < need) return QMOE_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return QMOE_ERR_ALIGN;
  }
  const int T = (int)indices->dims[0], k = (int)indices->dims[1];
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  int* inv = static_cast<int*>(const_cast<void*>(inverse->data));
  if (launch_sort_slots(indices->data, indices->dtype == QMOE_I64, T * k, (int)experts, static_cast<int*>(workspace),
                        static_cast<int*>(const_cast<void*>(offsets->data)),
                        perm ? static_cast<int*>(const_cast<void*>(perm->data)) : nullptr, inv, s) != hipSuccess)
    return QMOE_ERR_HIP;
  if (numel(rows) > 0 && launch_dispatch_rows(row_type(input->dtype), input->data, inv, T, k, input->dims[1],
                                              const_cast<void*>(rows->data), s) != hipSuccess)
    return QMOE_ERR_HIP;
  return QMOE_OK;
}

qmoe_status qmoe_dispatch_backward(const qmoe_tensor* grad_rows, const qmoe_tensor* inverse,
                                   const qmoe_tensor* grad_input, void* stream) {
  return qmoe_combine(grad_rows, inverse, nullptr, grad_input, stream);
}

qmoe_status qmoe_combine(const qmoe_tensor* rows, const qmoe_tensor* inverse, const qmoe_tensor* weights,
                         const qmoe_tensor* output, void* stream) {
  if (!rows || !inverse || !output) return QMOE_ERR_NULL;
  qmoe_status st = check_rows(inverse, {rows}, {output});
  if (st != QMOE_OK) return st;
  const int64_t T = inverse->dims[0], k = inverse->dims[1], H = output->dims[1];
  if (weights && weights->dtype != QMOE_F32) return QMOE_ERR_DTYPE;
  if (weights && !is(weights, {T, k})) return QMOE_ERR_SHAPE;
  if (row_too_long(H)) return QMOE_ERR_UNSUPPORTED;
  if (T == 0 || H == 0) return QMOE_OK;
  st = check_data({rows, inverse, weights, output});
  if (st != QMOE_OK) return st;
  return launch_combine_rows(row_type(rows->dtype), rows->data, static_cast<const int*>(inverse->data),
                             weights ? static_cast<const float*>(weights->data) : nullptr, (int)T, (int)k, H,
                             const_cast<void*>(output->data), reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? QMOE_OK
             : QMOE_ERR_HIP;
}

qmoe_status qmoe_combine_backward(const qmoe_tensor* grad_output, const qmoe_tensor* rows, const qmoe_tensor* inverse,
                                  const qmoe_tensor* weights, const qmoe_tensor* grad_rows,
                                  const qmoe_tensor* grad_weights, void* stream) {
  if (!grad_output || !rows || !inverse || !weights) return QMOE_ERR_NULL;
  qmoe_status st = check_rows(inverse, {rows, grad_rows}, {grad_output});
  if (st != QMOE_OK) return st;
  const int64_t T = inverse->dims[0], k = inverse->dims[1], H = rows->dims[1];
  if (weights->dtype != QMOE_F32 || (grad_weights && grad_weights->dtype != QMOE_F32)) return QMOE_ERR_DTYPE;
  if (!is(weights, {T, k}) || (grad_weights && !is(grad_weights, {T, k}))) return QMOE_ERR_SHAPE;
  if (row_too_long(H)) return QMOE_ERR_UNSUPPORTED;
  if (T * k == 0 || (!grad_rows && !grad_weights)) return QMOE_OK;
  st = check_data({grad_output, rows, inverse, weights, grad_rows, grad_weights});
  if (st != QMOE_OK) return st;
  return launch_combine_grad(row_type(rows->dtype), grad_output->data, rows->data,
                             static_cast<const int*>(inverse->data), static_cast<const float*>(weights->data), (int)T,
                             (int)k, H, grad_rows ? const_cast<void*>(grad_rows->data) : nullptr,
                             grad_weights ? static_cast<float*>(const_cast<void*>(grad_weights->data)) : nullptr,
                             reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? QMOE_OK
             : QMOE_ERR_HIP;
}

}  // extern "C"
