// Routing from scores with a balance bias and groups of experts, and its
// gradient: launch functions (host side; enqueue only).
#pragma once
#include <hip/hip_runtime.h>

namespace qmoe {

struct RouteScored {
  int E, k;
  int sigmoid;          // 0: softmax over all unmasked experts
  int groups, kept;     // groups of E / groups consecutive experts, kept of them selected from
  int group_top;        // 1 or 2: a group is ranked by the sum of so many of its largest
  int normalize;
  float scale;
};
constexpr int kMaxRouteGroups = 64;

// bias [E] or NULL.
hipError_t launch_route_scored(const float* logits, const float* bias, int T, const RouteScored& a, int* idx, float* w,
                               hipStream_t st);
hipError_t launch_route_scored_grad(const float* gw, const float* logits, const void* idx, bool idx64, int T,
                                    const RouteScored& a, float* gl, hipStream_t st);

}  // namespace qmoe
