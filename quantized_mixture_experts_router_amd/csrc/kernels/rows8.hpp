// Device helpers of rows held in 8 bits (rows8.h).
//
// A block of a row's columns shares a scale 2^e; with m the block's largest
// magnitude, e is the least integer (at least -126) with
//   int8   m <  127.5 2^e    code rint(v 2^-e) + 128, 1 .. 255
//   e4m3   m <= 464 2^e      code v 2^-e rounded to that type (464 is the last value that rounds to its largest, 448)
// and 0 for a block of zeros.  A power of two makes v 2^-e exact, so a code
// carries one rounding (half a step of 2^e; for e4m3 2^-4 of the value, or half
// a subnormal step, 2^-10 2^e), and the values a code stands for (at most eight
// significant bits) exact in every row type.  A NaN or an infinity makes the scale
// NaN and with it every value of its block.
#pragma once
#include <type_traits>

#include "rows8.h"
#include "wave.hpp"

namespace qmoe {

// Bits of the scale from the bits of m (which order like the magnitudes, NaN above infinity).
__device__ __forceinline__ uint32_t r8_scale_bits(int format, uint32_t m) {
  // m = 2^x 1.f: e = x - 6 unless 1.f >= 1.9921875 (int8), x - 8 unless 1.f > 1.8125 (e4m3): the sum carries into the exponent then
  const uint32_t carry = format == R8_INT8 ? 0x010000u : 0x17ffffu;
  const int below = format == R8_INT8 ? 6 : 8;
  uint32_t s = (uint32_t)max((int)((m + carry) >> 23) - below, 1) << 23;
  s = m == 0u ? 0x3f800000u : s;
  return m >= 0x7f800000u ? 0x7fc00000u : s;
}
template <int F>
__device__ __forceinline__ uint32_t r8_scale_bits(uint32_t m) {
  return r8_scale_bits(F, m);
}
// 1 / scale (any number where that is NaN: whatever the codes are, their values are NaN).
__device__ __forceinline__ float r8_inverse(uint32_t scale_bits) { return __uint_as_float(0x7f000000u - scale_bits); }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Largest of the 2^log lanes that differ in the low bits (log uniform, up to 6; every lane active).
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int log) {
  if (log > 0) v = max(v, dpp_from<kDppXor1>(v));
  if (log > 1) v = max(v, dpp_from<kDppXor2>(v));
  if (log > 2) v = max(v, dpp_from<kDppHalf>(v));
  if (log > 3) v = max(v, dpp_from<kDppRow>(v));
  if (log > 4) {
    uint32_t o = v;
    swap16(v, o);
    v = max(v, o);
  }
  if (log > 5) {
    uint32_t o = v;
    swap32(v, o);
    v = max(v, o);
  }
  return v;
}

// Four codes of v * inv, the first in the low byte.
template <int F>
__device__ __forceinline__ uint32_t r8_encode4(float a, float b, float c, float d, float inv) {
  if constexpr (F == R8_INT8) {
    // 1.5 2^23 + 128 + q rounds q to an integer, ties to even, and leaves its code in the low byte
    const float mid = 12583040.f;
    const uint32_t x = __float_as_uint(fmaf(a, inv, mid)), y = __float_as_uint(fmaf(b, inv, mid));
    const uint32_t z = __float_as_uint(fmaf(c, inv, mid)), w = __float_as_uint(fmaf(d, inv, mid));
    const uint32_t lo = __builtin_amdgcn_perm(y, x, 0x0c0c0400u), hi = __builtin_amdgcn_perm(w, z, 0x04000c0cu);
    return lo | hi;
  } else {
    int u = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, u, true);
  }
}

// The values of four codes.
template <int F>
__device__ __forceinline__ void r8_decode4(uint32_t u, float scale, float* v) {
  if constexpr (F == R8_INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ((float)((u >> (8 * i)) & 0xffu) - 128.f) * scale;
  } else {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)u, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)u, true);
    v[0] = lo[0] * scale;
    v[1] = lo[1] * scale;
    v[2] = hi[0] * scale;
    v[3] = hi[1] * scale;
  }
}

// Values beyond the largest finite one of the type become it (the rounding to
// codes can pass it where the block reaches the type's top); NaN stays.
template <typename ET>
__device__ __forceinline__ float r8_limit(float v) {
  constexpr float top = std::is_same<ET, _Float16>::value ? 65504.f : std::is_same<ET, float>::value ? 3.4028234664e38f : 3.3895313892515355e38f;
  v = v > top ? top : v;
  return v < -top ? -top : v;
}
// Scales below it: no code passes the type's range.
template <typename ET, int F>
__device__ __forceinline__ bool r8_may_pass(float scale) {
  constexpr float from = std::is_same<ET, _Float16>::value ? (F == R8_INT8 ? 1024.f : 256.f)
                                                           : (F == R8_INT8 ? 0x1p122f : 0x1p120f);
  return fabsf(scale) >= from;
}

// W consecutive elements of a row of which n are left, at element alignment
// (the hardware takes wide accesses at any address): one access where all are
// there; zeros past the row's end.
template <typename ET, int W>
struct RowPiece {
  typedef ET type __attribute__((ext_vector_type(W)));
  typedef type any __attribute__((aligned(sizeof(ET))));
};
template <typename ET, int W>
__device__ __forceinline__ typename RowPiece<ET, W>::type load_piece(const ET* p, int n) {
  typename RowPiece<ET, W>::type t = {};
  if (n >= W) return *(const typename RowPiece<ET, W>::any*)p;
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (i < n) t[i] = p[i];
  return t;
}
// stream (uniform): past the caches.
template <typename ET, int W>
__device__ __forceinline__ void store_piece(ET* p, int n, typename RowPiece<ET, W>::type t, int stream = 0) {
  if (n >= W) {
    if (stream) {
      asm volatile("");  // (the compiler would make one plain store of both branches')
      __builtin_nontemporal_store(t, (typename RowPiece<ET, W>::any*)p);
      asm volatile("");
    } else *(typename RowPiece<ET, W>::any*)p = t;
    return;
  }
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (i < n) p[i] = t[i];
}

template <int F>
__device__ __forceinline__ uint32_t r8_encode4(const f32x4& v, float inv) {
  return r8_encode4<F>(v[0], v[1], v[2], v[3], inv);
}

// Codes of W (2, 4 or 8) values behind p, n of them in the row.
template <int F, int W>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, const float (&v)[W], float inv) {
  uint32_t u[(W + 3) / 4];
  if constexpr (W == 2) u[0] = r8_encode4<F>(v[0], v[1], 0.f, 0.f, inv);
#pragma unroll
  for (int i = 0; i < W / 4; ++i) u[i] = r8_encode4<F>(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], inv);
  typename RowPiece<uint8_t, W>::type t;
  __builtin_memcpy(&t, u, W);
  store_piece<uint8_t, W>(p, n, t);
}
// Values of the W codes behind p, n of them in the row (zeros past its end),
// within the range of ET.
template <typename ET, int F, int W>
__device__ __forceinline__ void load_codes(const uint8_t* p, int n, float scale, float (&v)[W]) {
  const auto t = load_piece<uint8_t, W>(p, n);
  uint32_t u[W / 4];
  __builtin_memcpy(u, &t, W);
#pragma unroll
  for (int i = 0; i < W / 4; ++i) r8_decode4<F>(u[i], scale, v + 4 * i);
  if (r8_may_pass<ET, F>(scale)) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = r8_limit<ET>(v[i]);
  }
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = i < n ? v[i] : 0.f;
}

// f(format) with the format as a compile-time constant.
template <typename G>
__host__ __device__ __forceinline__ void with_format(int format, G f) {
  if (format == R8_INT8) f(std::integral_constant<int, R8_INT8>{});
  else f(std::integral_constant<int, R8_E4M3>{});
}

}  // namespace qmoe
