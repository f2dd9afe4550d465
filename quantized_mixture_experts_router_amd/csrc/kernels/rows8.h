// Rows held in 8 bits with a power-of-two scale per block of columns: launch
// functions (host side; enqueue only).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmoe {

enum Rows8Format { R8_INT8 = 0, R8_E4M3 = 1 };

// Codes [rows][cols] and scales [rows][ceil(cols / block)] of one format; block
// = 1 << block_log columns, 16 .. 128.
struct Rows8 {
  uint8_t* codes;
  float* scales;
  int format, block_log;
};

hipError_t launch_quantize_rows(int type, const void* x, long M, long N, const Rows8& q, hipStream_t st);

// out[m] = the values of row m, or (perm) of row perm[m] / k (entries outside
// [0, M): zeros), rows of ld >= N elements, zeros from N on.  M: rows of out.
// soon: the caller reads them right away, they stay in the caches whatever their size.
hipError_t launch_dequantize_rows(int type, const Rows8& q, const int* perm, int k, long M, long N, void* out, long ld,
                                  bool soon, hipStream_t st);

}  // namespace qmoe
