// The linear layers' matrix kernel on bf16 operands (linear_kernel.hpp).
#include "linear_kernel.hpp"

namespace qmoe {
hipError_t launch_linear_bf16(int mode, int tile, const LinearGemm& g, hipStream_t st) {
  return go_mode<__bf16>(mode, tile, g, st);
}
}  // namespace qmoe
