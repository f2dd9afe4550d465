// C ABI of the root-mean-square norm (declared in include/qmoe.h): contract
// checks and enqueue.
#include <hip/hip_runtime.h>

#include "kernels/norm.h"
#include "qmoe_checks.h"

using namespace qmoe;

namespace {

// rows [M, H] of one type, weight [H] of it or NULL; any of rows but the first may be NULL.
qmoe_status check_norm(std::initializer_list<const qmoe_tensor*> rows, const qmoe_tensor* weight, float epsilon) {
  const qmoe_tensor* first = *rows.begin();
  for (const qmoe_tensor* t : rows)
    if (t && (t->rank != 2 || t->dims[0] < 0 || t->dims[1] < 0)) return QMOE_ERR_SHAPE;
  if (weight && weight->rank != 1) return QMOE_ERR_SHAPE;
  if (!float_code(first->dtype)) return QMOE_ERR_DTYPE;
  for (const qmoe_tensor* t : rows)
    if (t && t->dtype != first->dtype) return QMOE_ERR_DTYPE;
  if (weight && weight->dtype != first->dtype) return QMOE_ERR_DTYPE;
  if (!(epsilon > 0.f && epsilon <= 3.4028234664e38f)) return QMOE_ERR_ATTR;
  for (const qmoe_tensor* t : rows)
    if (t && !is(t, {first->dims[0], first->dims[1]})) return QMOE_ERR_SHAPE;
  if (weight && weight->dims[0] != first->dims[1]) return QMOE_ERR_SHAPE;
  if (first->dims[0] > kMaxRowCount || first->dims[1] > kMaxRowCols) return QMOE_ERR_UNSUPPORTED;
  return QMOE_OK;
}

qmoe_status check_norm_grads(const qmoe_tensor* grad_output, const qmoe_tensor* grad_sum, const qmoe_tensor* input,
                             const qmoe_tensor* weight, float epsilon, const qmoe_tensor* grad_input,
                             const qmoe_tensor* grad_weight, size_t* bytes) {
  if (!grad_output || !input) return QMOE_ERR_NULL;
  if (grad_weight && !weight) return QMOE_ERR_NULL;
  qmoe_status st = check_norm({grad_output, grad_sum, input, grad_input}, weight, epsilon);
  if (st != QMOE_OK) return st;
  if (grad_weight && grad_weight->dtype != input->dtype) return QMOE_ERR_DTYPE;
  if (grad_weight && !is(grad_weight, {input->dims[1]})) return QMOE_ERR_SHAPE;
  *bytes = grad_weight ? sizeof(float) * norm_partials(row_type(input->dtype), input->dims[0], input->dims[1]) : 0;
  return QMOE_OK;
}

}  // namespace

extern "C" {

qmoe_status qmoe_rms_norm(const qmoe_tensor* input, const qmoe_tensor* residual, const qmoe_tensor* weight,
                          float epsilon, const qmoe_tensor* sum, const qmoe_tensor* output, const qmoe_tensor* codes,
                          const qmoe_tensor* scales, int64_t block_size, void* stream) {
  if (!input || (!output && !codes) || (sum && !residual) || (codes == nullptr) != (scales == nullptr))
    return QMOE_ERR_NULL;
  qmoe_status st = check_norm({input, residual, sum, output}, weight, epsilon);
  if (st == QMOE_OK && codes) st = check_rows8(codes, scales, input->dims[0], input->dims[1], block_size);
  if (st != QMOE_OK) return st;
  if (input->dims[0] == 0 || input->dims[1] == 0) return QMOE_OK;
  st = check_data({input, residual, weight, sum, output, codes, scales});
  if (st != QMOE_OK) return st;
  Norm a{};
  a.x = input->data;
  a.r = data_of(residual);
  a.w = data_of(weight);
  a.sum = data_of(sum);
  a.y = data_of(output);
  if (codes) a.q = rows8_of(codes, scales, block_size);
  a.M = input->dims[0];
  a.H = (int)input->dims[1];
  a.eps = epsilon;
  return launch_rms_norm(row_type(input->dtype), a, reinterpret_cast<hipStream_t>(stream)) == hipSuccess ? QMOE_OK
                                                                                                        : QMOE_ERR_HIP;
}

qmoe_status qmoe_rms_norm_backward_workspace_size(const qmoe_tensor* grad_output, const qmoe_tensor* grad_sum,
                                                  const qmoe_tensor* input, const qmoe_tensor* weight, float epsilon,
                                                  const qmoe_tensor* grad_input, const qmoe_tensor* grad_weight,
                                                  size_t* bytes) {
  if (!bytes) return QMOE_ERR_NULL;
  return check_norm_grads(grad_output, grad_sum, input, weight, epsilon, grad_input, grad_weight, bytes);
}

qmoe_status qmoe_rms_norm_backward(const qmoe_tensor* grad_output, const qmoe_tensor* grad_sum,
                                   const qmoe_tensor* input, const qmoe_tensor* weight, float epsilon,
                                   const qmoe_tensor* grad_input, const qmoe_tensor* grad_weight, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  size_t need = 0;
  qmoe_status st = check_norm_grads(grad_output, grad_sum, input, weight, epsilon, grad_input, grad_weight, &need);
  if (st != QMOE_OK) return st;
  const int64_t M = input->dims[0], H = input->dims[1];
  if (H == 0 || (M == 0 && !grad_weight) || (!grad_input && !grad_weight)) return QMOE_OK;
  st = check_data({grad_output, grad_sum, input, weight, grad_input, grad_weight});
  if (st == QMOE_OK) st = check_ws(workspace, workspace_bytes, need);
  if (st != QMOE_OK) return st;
  NormGrad a{};
  a.dy = grad_output->data;
  a.ds = data_of(grad_sum);
  a.h = input->data;
  a.w = data_of(weight);
  a.dh = data_of(grad_input);
  a.dw = data_of(grad_weight);
  a.partial = static_cast<float*>(workspace);
  a.M = M;
  a.H = (int)H;
  a.eps = epsilon;
  return launch_rms_norm_grad(row_type(input->dtype), a, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? QMOE_OK
             : QMOE_ERR_HIP;
}

}  // extern "C"
