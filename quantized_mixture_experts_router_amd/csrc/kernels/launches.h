// Launches of more workgroups than one dimension of a grid holds threads for.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>

namespace qmoe {

// One dimension of a launch holds fewer than 2^32 threads (beyond, a launch
// covers only a part and reports success): `blocks` workgroups of up to 512
// threads in launches of 2^22 at most, f(first, count) each.
constexpr long kMaxLaunch = 1l << 22;
template <typename F>
hipError_t in_launches(long blocks, F f) {
  for (long b = 0; b < blocks; b += kMaxLaunch) {
    f((int)b, (unsigned)std::min(blocks - b, kMaxLaunch));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qmoe
