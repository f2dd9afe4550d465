// Device helpers of the linear layers: activations and their derivatives,
// and the walk from a row-block index to its group.
#pragma once
#include <math.h>

#include "common.hpp"
#include "linear.h"

namespace qmoe {

typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Activation codes (qmoe_activation of include/qmoe.h).
constexpr int kActRelu = 0, kActSwiglu = 1, kActGelu = 2, kActSilu = 3, kActIdentity = 4;

// 1 / (1 + e^-v), finite for every v: e^-v may overflow to infinity, whose
// reciprocal is the right 0.
__device__ __forceinline__ float lin_sigmoid(float v) { return 1.f / (1.f + expf(-v)); }

__device__ __forceinline__ float lin_act(float z, const LinearAct& a) {
  if (a.type == kActRelu) return z < 0.f ? 0.f : z;  // NaN stays NaN
  if (a.type == kActGelu) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  if (a.type == kActSilu) return z * lin_sigmoid(z);
  return z;
}

// g sigma(alpha g) (u + beta), with a limit L: g <- min(g, L), u <- clamp(u, -L, L)
__device__ __forceinline__ float lin_swiglu(float g, float u, const LinearAct& a) {
  if (a.has_limit) {
    g = g > a.limit ? a.limit : g;
    u = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
  }
  return g * lin_sigmoid(a.alpha * g) * (u + a.beta);
}

// d act / dz times dy
__device__ __forceinline__ float lin_act_grad(float dy, float z, const LinearAct& a) {
  if (a.type == kActRelu) return z > 0.f ? dy : 0.f;
  if (a.type == kActGelu) {
    const float cdf = 0.5f * (1.f + erff(z * 0.70710678118654752f));
    return dy * (cdf + z * 0.39894228040143268f * expf(-0.5f * z * z));
  }
  if (a.type == kActSilu) {
    const float s = lin_sigmoid(z);
    return dy * s * (1.f + z * (1.f - s));
  }
  return dy;
}

// Gradients at gate and linear branch; a clamped value passes none (at the
// bound itself it passes).
__device__ __forceinline__ void lin_swiglu_grad(float dy, float g, float u, const LinearAct& a, float& dg, float& du) {
  bool gp = true, up = true;
  if (a.has_limit) {
    gp = !(g > a.limit);
    up = !(u > a.limit || u < -a.limit);
    g = gp ? g : a.limit;
    u = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
  }
  const float s = lin_sigmoid(a.alpha * g);
  dg = gp ? dy * (u + a.beta) * s * (1.f + a.alpha * g * (1.f - s)) : 0.f;
  du = up ? dy * g * s : 0.f;
}

// Rows [lo, hi) of group g: the first group starts at row 0, and bounds
// outside [0, M] or falling are pulled back in, so that no offsets make an
// access leave the rows; g == G: the rows behind the last group.
__device__ __forceinline__ void group_rows(const int* __restrict__ offsets, int G, int M, int g, int& lo, int& hi) {
  if (!offsets) {
    lo = 0;
    hi = g == 0 ? M : 0;
    return;
  }
  lo = g == 0 ? 0 : min(max(offsets[g], 0), M);
  hi = g < G ? min(max(offsets[g + 1], lo), M) : M;
}

// Row block b (bm rows of one group each, the groups in order, then the rows
// behind the last group as group G): its group and rows [lo, hi) from the
// block's first row on (hi = the group's end).  False: past the last block.
// Every lane of a wavefront gets the same answer.
__device__ __forceinline__ bool find_block(const int* __restrict__ offsets, int G, int M, int bm, int b, int& g,
                                           int& lo, int& hi) {
  if (!offsets) {
    g = 0;
    lo = b * bm;
    hi = M;
    return lo < M;
  }
  const int lane = lane_id();
  int seen = 0;
  for (int c = 0; c <= G; c += 64) {
    int l = 0, h = 0;
    if (c + lane <= G) group_rows(offsets, G, M, c + lane, l, h);
    const int n = (h - l + bm - 1) / bm;
    int inc = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(inc, o);
      if (lane >= o) inc += v;
    }
    const unsigned long long past = __ballot(seen + inc > b);
    if (past) {
      const int f = __ffsll((long long)past) - 1;
      const int first = __shfl(seen + inc - n, f);
      g = __builtin_amdgcn_readfirstlane(c + f);
      lo = __builtin_amdgcn_readfirstlane(__shfl(l, f) + (b - first) * bm);
      hi = __builtin_amdgcn_readfirstlane(__shfl(h, f));
      return true;
    }
    seen += __shfl(inc, 63);
  }
  return false;
}

// First row block of group g (find_block's order) and its count of blocks.
__device__ __forceinline__ void group_blocks(const int* __restrict__ offsets, int G, int M, int bm, int g, int& first,
                                             int& count) {
  first = 0;
  count = 0;
  if (!offsets) {
    count = g == 0 ? (M + bm - 1) / bm : 0;
    return;
  }
  const int lane = lane_id();
  int sum = 0;
  for (int c = lane; c < g; c += 64) {
    int l, h;
    group_rows(offsets, G, M, c, l, h);
    sum += (h - l + bm - 1) / bm;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  first = sum;
  int l, h;
  group_rows(offsets, G, M, g, l, h);
  count = (h - l + bm - 1) / bm;
}

template <typename ET>
struct LinVec4 {
  typedef ET type __attribute__((ext_vector_type(4)));
};
template <typename ET>
struct LinVec2 {
  typedef ET type __attribute__((ext_vector_type(2)));
};

// The epilogue of four consecutive columns n .. n + 3 of output row m: z =
// the float32 sums, bias in, pre-activation out, activation, residual, one
// rounding to the type.  VEC: four columns at a time (N % 4 == 0 and pointers
// that allow it), else one by one up to N.
template <typename ET, bool VEC>
__device__ __forceinline__ void linear_epilogue(const LinearGemm& g, int grp, int m, int n, f32x4 z) {
  using V4 = typename LinVec4<ET>::type;
  using V2 = typename LinVec2<ET>::type;
  if (n >= g.N) return;
  const ET* bias = static_cast<const ET*>(g.bias);
  if constexpr (VEC) {
    if (bias) {
      const V4 b = *(const V4*)(bias + (long)grp * g.N + n);
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] += (float)b[i];
    }
    if (g.pre) {
      V4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (ET)z[i];
      *(V4*)(static_cast<ET*>(g.pre) + (long)m * g.N + n) = v;
    }
    if (g.act.type == kActSwiglu) {
      const long o = (long)m * (g.N >> 1) + (n >> 1);
      float y0 = lin_swiglu(z[0], z[1], g.act), y1 = lin_swiglu(z[2], z[3], g.act);
      if (g.res) {
        const V2 r = *(const V2*)(static_cast<const ET*>(g.res) + o);
        y0 += (float)r[0];
        y1 += (float)r[1];
      }
      V2 v;
      v[0] = (ET)y0;
      v[1] = (ET)y1;
      *(V2*)(static_cast<ET*>(g.out) + o) = v;
    } else {
      const long o = (long)m * g.N + n;
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = lin_act(z[i], g.act);
      if (g.res) {
        const V4 r = *(const V4*)(static_cast<const ET*>(g.res) + o);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] += (float)r[i];
      }
      V4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (ET)z[i];
      *(V4*)(static_cast<ET*>(g.out) + o) = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n + i >= g.N) continue;
      if (bias) z[i] += (float)bias[(long)grp * g.N + n + i];
      if (g.pre) static_cast<ET*>(g.pre)[(long)m * g.N + n + i] = (ET)z[i];
    }
    if (g.act.type == kActSwiglu) {
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        if (n + i >= g.N) continue;  // N is even: both or none
        const long o = (long)m * (g.N >> 1) + ((n + i) >> 1);
        float y = lin_swiglu(z[i], z[i + 1], g.act);
        if (g.res) y += (float)static_cast<const ET*>(g.res)[o];
        static_cast<ET*>(g.out)[o] = (ET)y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (n + i >= g.N) continue;
        const long o = (long)m * g.N + n + i;
        float y = lin_act(z[i], g.act);
        if (g.res) y += (float)static_cast<const ET*>(g.res)[o];
        static_cast<ET*>(g.out)[o] = (ET)y;
      }
    }
  }
}

// Zeros where the epilogue of the same columns would write (rows behind the
// last group).
template <typename ET>
__device__ __forceinline__ void linear_zero(const LinearGemm& g, int m, int n) {
  const bool glu = g.act.type == kActSwiglu;
  const long No = glu ? g.N >> 1 : g.N;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= g.N) continue;
    if (g.pre) static_cast<ET*>(g.pre)[(long)m * g.N + n + i] = (ET)0.f;
    if (!glu) static_cast<ET*>(g.out)[(long)m * No + n + i] = (ET)0.f;
    else if (i % 2 == 0) static_cast<ET*>(g.out)[(long)m * No + ((n + i) >> 1)] = (ET)0.f;
  }
}

// Four consecutive columns of a gradient row of `cols` columns.
template <typename ET, bool VEC>
__device__ __forceinline__ void store_cols4(ET* row, int c, int cols, f32x4 v) {
  if (c >= cols) return;
  if constexpr (VEC) {
    typename LinVec4<ET>::type t;
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = (ET)v[i];
    *(typename LinVec4<ET>::type*)(row + c) = t;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < cols) row[c + i] = (ET)v[i];
  }
}

// Four columns at a time where every row allows it.
template <typename ET>
bool linear_vec(const LinearGemm& g, int mode) {
  const uintptr_t a4 = 4 * sizeof(ET) - 1;
  auto al = [&](const void* p, uintptr_t m) { return (reinterpret_cast<uintptr_t>(p) & m) == 0; };
  if (mode != LIN_FWD) return g.K % 4 == 0 && al(g.out, a4);
  const uintptr_t ao = g.act.type == kActSwiglu ? 2 * sizeof(ET) - 1 : a4;
  return g.N % 4 == 0 && al(g.out, ao) && al(g.res, ao) && al(g.bias, a4) && al(g.pre, a4);
}

}  // namespace qmoe
