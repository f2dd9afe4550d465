// Root-mean-square norm of rows with the residual's addition, its output in
// the row type and / or in 8 bits, and its gradients: launch functions (host
// side; enqueue only).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rows8.h"

namespace qmoe {

//   h = x + r (rounded to the row type),  y = h w / sqrt(mean(h^2) + eps)
struct Norm {
  const void* x;  // [M][H]
  const void* r;  // [M][H] or NULL
  const void* w;  // [H] or NULL: 1
  void* sum;      // h [M][H] or NULL
  void* y;        // [M][H] or NULL
  Rows8 q;        // codes NULL: none
  long M;
  int H;
  int stream;     // outputs past the caches (set by the launch)
  float eps;
};
hipError_t launch_rms_norm(int type, const Norm& a, hipStream_t st);

//   dh = ds + s (dy w - n mean(dy w n)),  dw = sum_m dy n,  s = 1 / sqrt(mean(h^2) + eps),  n = s h
struct NormGrad {
  const void* dy;  // [M][H]
  const void* ds;  // [M][H] or NULL: gradient that arrives at h itself
  const void* h;   // [M][H]
  const void* w;   // [H] or NULL
  void* dh;        // [M][H] or NULL
  void* dw;        // [H] or NULL
  float* partial;  // norm_partials floats (dw)
  long M;
  int H;
  int stream;      // as above
  float eps;
};
// Floats of partial.
size_t norm_partials(int type, long M, long H);
hipError_t launch_rms_norm_grad(int type, const NormGrad& a, hipStream_t st);

}  // namespace qmoe
