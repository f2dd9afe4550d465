// Contract checks shared by the entry points on rows (host code).
#pragma once
#include <stdint.h>

#include <initializer_list>

#include "kernels/rows8.h"
#include "kernels/tokens.h"
#include "qmoe.h"

namespace qmoe {

inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int64_t numel(const qmoe_tensor* t) {
  int64_t n = 1;
  for (int i = 0; i < t->rank; ++i) n *= t->dims[i];
  return n;
}

inline bool is(const qmoe_tensor* t, std::initializer_list<int64_t> dims) {
  if (t->rank != (int)dims.size()) return false;
  int i = 0;
  for (int64_t d : dims)
    if (t->dims[i++] != d) return false;
  return true;
}

inline bool float_code(int32_t dt) { return dt == QMOE_F32 || dt == QMOE_F16 || dt == QMOE_BF16; }
inline bool index_code(int32_t dt) { return dt == QMOE_I32 || dt == QMOE_I64; }
inline bool eight_code(int32_t dt) { return dt == QMOE_U8 || dt == QMOE_E4M3; }
inline int row_type(int32_t dt) { return dt == QMOE_F32 ? ROW_F32 : dt == QMOE_F16 ? ROW_F16 : ROW_BF16; }
inline uintptr_t esize(int32_t dt) {
  switch (dt) {
    case QMOE_U8:
    case QMOE_E4M3: return 1;
    case QMOE_F16:
    case QMOE_BF16: return 2;
    case QMOE_I64:
    case QMOE_F64: return 8;
  }
  return 4;
}

// Pointers present where there are elements, aligned to the element.
inline qmoe_status check_data(std::initializer_list<const qmoe_tensor*> ts) {
  for (const qmoe_tensor* t : ts) {
    if (!t) continue;
    if (numel(t) > 0 && !t->data) return QMOE_ERR_NULL;
    if (!aligned_to(t->data, esize(t->dtype))) return QMOE_ERR_ALIGN;
  }
  return QMOE_OK;
}

inline qmoe_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return QMOE_OK;
  if (!ws) return QMOE_ERR_NULL;
  if (have < need) return QMOE_ERR_WORKSPACE;
  return aligned_to(ws, 256) ? QMOE_OK : QMOE_ERR_ALIGN;
}

constexpr int64_t kMaxRowCols = int64_t(1) << 20;   // columns of a row
constexpr int64_t kMaxRowCount = int64_t(1) << 30;  // rows

// log2 of a block size of rows in 8 bits, or -1.
inline int block_log(int64_t block_size) {
  for (int l = 4; l <= 7; ++l)
    if (block_size == int64_t(1) << l) return l;
  return -1;
}

// codes and scales of M rows of N columns (both given): types, then shapes.
inline qmoe_status check_rows8(const qmoe_tensor* codes, const qmoe_tensor* scales, int64_t M, int64_t N,
                               int64_t block_size) {
  if (!codes || !scales) return QMOE_ERR_NULL;
  if (!eight_code(codes->dtype) || scales->dtype != QMOE_F32) return QMOE_ERR_DTYPE;
  if (block_log(block_size) < 0) return QMOE_ERR_ATTR;
  if (!is(codes, {M, N}) || !is(scales, {M, (N + block_size - 1) / block_size})) return QMOE_ERR_SHAPE;
  return QMOE_OK;
}

inline Rows8 rows8_of(const qmoe_tensor* codes, const qmoe_tensor* scales, int64_t block_size) {
  return {static_cast<uint8_t*>(const_cast<void*>(codes->data)), static_cast<float*>(const_cast<void*>(scales->data)),
          codes->dtype == QMOE_U8 ? R8_INT8 : R8_E4M3, block_log(block_size)};
}

inline void* data_of(const qmoe_tensor* t) { return t ? const_cast<void*>(t->data) : nullptr; }

}  // namespace qmoe
