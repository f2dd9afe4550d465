// Reductions over the 64 lanes of a wavefront in registers (no LDS): the lanes
// of a row of 16 exchange by DPP, the rows by row swaps.  Every lane gets the
// result; every lane has to be active.
#pragma once
#include "common.hpp"

namespace qmoe {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_from(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
constexpr int kDppXor1 = 0xb1, kDppXor2 = 0x4e;  // quad_perm [1, 0, 3, 2], [2, 3, 0, 1]
constexpr int kDppHalf = 0x141, kDppRow = 0x140;  // mirrors of eight and of sixteen lanes: the other half's values

// f(a, b) over all lanes of a 32-bit value.
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, F f) {
  v = f(v, dpp_from<kDppXor1>(v));
  v = f(v, dpp_from<kDppXor2>(v));
  v = f(v, dpp_from<kDppHalf>(v));
  v = f(v, dpp_from<kDppRow>(v));
  uint32_t a = v, b = v;
  swap16(a, b);
  v = f(a, b);
  a = b = v;
  swap32(a, b);
  return f(a, b);
}
__device__ __forceinline__ int wave_max_int(int v) {
  return (int)wave_reduce((uint32_t)v, [](uint32_t a, uint32_t b) { return (uint32_t)max((int)a, (int)b); });
}
__device__ __forceinline__ float wave_sum_float(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint64_t o = (uint64_t)dpp_from<CTRL>((uint32_t)(u >> 32)) << 32 | dpp_from<CTRL>((uint32_t)u);
  return v + __builtin_bit_cast(double, o);
}
// Sum over 8, 16, 32 or 64 lanes that differ in the low bits of their number.
template <int LANES = 64>
__device__ __forceinline__ double wave_sum_double(double v) {
  v = dpp_add<kDppXor1>(v);
  v = dpp_add<kDppXor2>(v);
  v = dpp_add<kDppHalf>(v);
  if constexpr (LANES > 8) v = dpp_add<kDppRow>(v);
  auto halves = [](double x, auto swap) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    uint32_t al = (uint32_t)u, ah = (uint32_t)(u >> 32), bl = al, bh = ah;
    swap(al, bl);
    swap(ah, bh);
    return __builtin_bit_cast(double, (uint64_t)ah << 32 | al) + __builtin_bit_cast(double, (uint64_t)bh << 32 | bl);
  };
  if constexpr (LANES > 16) v = halves(v, [](uint32_t& a, uint32_t& b) { swap16(a, b); });
  if constexpr (LANES > 32) v = halves(v, [](uint32_t& a, uint32_t& b) { swap32(a, b); });
  return v;
}

}  // namespace qmoe
