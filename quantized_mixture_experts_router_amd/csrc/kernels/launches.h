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

// A pass that writes this much (what the eight L2 caches hold) stores its rows past
// the caches: 4096 x 14336 from 8 bits to bfloat16 27 us (39 through them), a norm of
// 8192 x 4096 with residual 48 (50).  Smaller rows are read again from the caches (4096 x
// 4096 to 8 bits and back 18.8 us, 21.3 past them), and so are 8-bit codes of any size
// by what follows: 4096 x 14336 to 8 bits and back 31 and 28 us, 33 and 38 with the
// codes past them, a norm of 8192 x 4096 with 8 bits and their values 54 and 18, 58
// and 23.  Read much later, with 1 GiB read between, they lose nothing: 31 and 36 us
// against 33 and 36, 53 and 21 against 57 and 21.  (The codes that leave in a matrix
// product's epilogue go the way of its output.)
constexpr long kStreamBytes = 32l << 20;

}  // namespace qmoe
