// C ABI of rows held in 8 bits (declared in include/qmoe.h): contract checks
// and enqueue.
#include <hip/hip_runtime.h>

#include "qmoe_checks.h"

using namespace qmoe;

extern "C" {

qmoe_status qmoe_quantize_rows(const qmoe_tensor* input, int64_t block_size, const qmoe_tensor* codes,
                               const qmoe_tensor* scales, void* stream) {
  if (!input || !codes || !scales) return QMOE_ERR_NULL;
  if (input->rank != 2 || input->dims[0] < 0 || input->dims[1] < 0) return QMOE_ERR_SHAPE;
  if (!float_code(input->dtype)) return QMOE_ERR_DTYPE;
  const int64_t M = input->dims[0], N = input->dims[1];
  qmoe_status st = check_rows8(codes, scales, M, N, block_size);
  if (st != QMOE_OK) return st;
  if (M > kMaxRowCount || N > kMaxRowCols) return QMOE_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return QMOE_OK;
  st = check_data({input, codes, scales});
  if (st != QMOE_OK) return st;
  return launch_quantize_rows(row_type(input->dtype), input->data, M, N, rows8_of(codes, scales, block_size),
                              reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? QMOE_OK
             : QMOE_ERR_HIP;
}

qmoe_status qmoe_dequantize_rows(const qmoe_tensor* codes, const qmoe_tensor* scales, int64_t block_size,
                                 const qmoe_tensor* perm, const qmoe_tensor* output, void* stream) {
  if (!codes || !scales || !output) return QMOE_ERR_NULL;
  if (codes->rank != 2 || codes->dims[0] < 0 || codes->dims[1] < 0) return QMOE_ERR_SHAPE;
  if (output->rank != 2 || output->dims[0] < 0 || (perm && perm->rank != 1)) return QMOE_ERR_SHAPE;
  const int64_t T = codes->dims[0], N = codes->dims[1], M = output->dims[0];
  qmoe_status st = check_rows8(codes, scales, T, N, block_size);
  if (st != QMOE_OK) return st;
  if (!float_code(output->dtype) || (perm && perm->dtype != QMOE_I32)) return QMOE_ERR_DTYPE;
  if (output->dims[1] != N || (perm ? perm->dims[0] != M || (T == 0 ? M != 0 : M % T != 0) : M != T)) return QMOE_ERR_SHAPE;
  if (M > kMaxRowCount || T > kMaxRowCount || N > kMaxRowCols) return QMOE_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return QMOE_OK;
  st = check_data({codes, scales, perm, output});
  if (st != QMOE_OK) return st;
  return launch_dequantize_rows(row_type(output->dtype), rows8_of(codes, scales, block_size),
                                perm ? static_cast<const int*>(perm->data) : nullptr, (int)(M / T), M, N,
                                data_of(output), N, false, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? QMOE_OK
             : QMOE_ERR_HIP;
}

}  // extern "C"
