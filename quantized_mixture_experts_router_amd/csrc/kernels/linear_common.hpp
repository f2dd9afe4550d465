// Device helpers of the linear layers: activations and their derivatives,
// and the walk from a row-block index to its group.
#pragma once
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "linear.h"
#include "linear_tiles.h"
#include "rows8.hpp"

namespace qmoe {

typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Activation codes (qmoe_activation of include/qmoe.h).
constexpr int kActRelu = 0, kActSwiglu = 1, kActGelu = 2, kActSilu = 3, kActIdentity = 4;

// 1 / (1 + e^-v), finite for every v: e^-v may overflow to infinity, whose
// reciprocal is the right 0.  FAST (results that are rounded to 16 bits): the
// hardware's exponential and reciprocal, each within 2^-22 of 1 relative and
// |v| 2^-24 for the argument's scaling, far below half a step of the types
// (2^-11, 2^-8); the full ones made the epilogue of a 256 x 256 SwiGLU tile 9 us
// of arithmetic and bound the activation's gradient pass.
template <bool FAST>
__device__ __forceinline__ float lin_sigmoid(float v) {
  if constexpr (FAST) return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
  return 1.f / (1.f + expf(-v));
}

// The normal distribution Phi(z) and e = exp(-z^2 / 2).  Below 0 it is taken
// as its own tail (1 + erf has lost 4 % of it at -5 and all of it at -5.6).
// FAST: the tail is e times a polynomial in t = 1 / (1 + 0.3 |z|) (a fit of
// Phi(-a) exp(a^2 / 2) over a in [0, 14], within 2^-22 relative), with the
// hardware's exponential and reciprocal as above: 2^-20 in all, and z^2 2^-24
// for the exponent's rounding, below 2^-9 of half a step of the 16-bit types.
// Forward of 8192 x 1024 -> 4096 float16 84 us (105 us with erfcf, 93 us with
// 1 + erff), the gradient's pass alone 42 us (70 and 52 us).
struct LinPhi {
  float phi, e;
};
template <bool FAST>
__device__ __forceinline__ LinPhi lin_phi(float z) {
  if constexpr (!FAST) return {0.5f * erfcf(z * -0.70710678118654752f), expf(-0.5f * z * z)};
  const float e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.3f, 1.f));
  float p = 0.03567499294877052f;
  p = fmaf(p, t, -0.15720391273498535f);
  p = fmaf(p, t, 0.20635481178760529f);
  p = fmaf(p, t, -0.053684744983911514f);
  p = fmaf(p, t, 0.12856215238571167f);
  p = fmaf(p, t, 0.0999133437871933f);
  p = fmaf(p, t, 0.12075397372245789f);
  p = fmaf(p, t, 0.11962930113077164f);
  const float tail = p * t * e;
  return {z > 0.f ? 1.f - tail : tail, e};
}

template <bool FAST>
__device__ __forceinline__ float lin_act(float z, int act) {
  if (act == kActRelu) return z < 0.f ? 0.f : z;  // NaN stays NaN
  if (act == kActGelu) return z * lin_phi<FAST>(z).phi;
  if (act == kActSilu) return z * lin_sigmoid<FAST>(z);
  return z;
}

// g sigma(alpha g) (u + beta), with a limit L: g <- min(g, L), u <- clamp(u, -L, L)
template <bool FAST>
__device__ __forceinline__ float lin_swiglu(float g, float u, const LinearAct& a) {
  if (a.has_limit) {
    g = g > a.limit ? a.limit : g;
    u = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
  }
  return g * lin_sigmoid<FAST>(a.alpha * g) * (u + a.beta);
}

// d act / dz times dy
template <bool FAST>
__device__ __forceinline__ float lin_act_grad(float dy, float z, int act) {
  if (act == kActRelu) return z > 0.f ? dy : 0.f;
  if (act == kActGelu) {
    const LinPhi n = lin_phi<FAST>(z);
    return dy * (n.phi + z * 0.39894228040143268f * n.e);
  }
  if (act == kActSilu) {
    const float s = lin_sigmoid<FAST>(z);
    return dy * s * (1.f + z * (1.f - s));
  }
  return dy;
}

// Gradients at gate and linear branch; a clamped value passes none (at the
// bound itself it passes).
template <bool FAST>
__device__ __forceinline__ void lin_swiglu_grad(float dy, float g, float u, const LinearAct& a, float& dg, float& du) {
  bool gp = true, up = true;
  if (a.has_limit) {
    gp = !(g > a.limit);
    up = !(u > a.limit || u < -a.limit);
    g = gp ? g : a.limit;
    u = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
  }
  const float s = lin_sigmoid<FAST>(a.alpha * g);
  // (alpha after g sigma (1 - sigma), which is small: alpha g alone may pass the largest float)
  dg = gp ? dy * (u + a.beta) * (s + a.alpha * (g * s * (1.f - s))) : 0.f;
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

// The rows of up to G + 1 groups (group G: the rows behind the last) as blocks
// of bm rows of one group each, in group order.  Every lane of a wavefront gets
// the same answers; groups 0 .. 63 stay in registers, a lane each.
struct RowBlocks {
  const int* offsets;
  int G, M, bm;
  int lo, n, inc;  // lane's group of the first 64: first row, blocks, blocks up to its end
  int hi;
  int total;       // blocks in all

  __device__ __forceinline__ void scan(int g, int& l, int& h, int& c, int& i) const {
    l = h = 0;
    if (g <= G) group_rows(offsets, G, M, g, l, h);
    c = (h - l + bm - 1) / bm;
    i = c;
    const int lane = lane_id();
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(i, o);
      if (lane >= o) i += v;
    }
  }
  __device__ __forceinline__ RowBlocks(const int* __restrict__ offs, int g, int m, int b)
      : offsets(offs), G(g), M(m), bm(b) {
    if (!offsets) {
      total = (M + bm - 1) / bm;
      return;
    }
    scan(lane_id(), lo, hi, n, inc);
    total = __builtin_amdgcn_readlane(inc, 63);
    for (int c = 64; c <= G; c += 64) {
      int l, h, k, i;
      scan(c + lane_id(), l, h, k, i);
      total += __builtin_amdgcn_readlane(i, 63);
    }
  }
  // Block b: its group and rows [l, h) from the block's first row on (h = the
  // group's end).  False: past the last block.
  __device__ __forceinline__ bool find(int b, int& g, int& l, int& h) const {
    if (b >= total) return false;
    if (!offsets) {
      g = 0;
      l = b * bm;
      h = M;
      return true;
    }
    int seen = 0, cl = lo, ch = hi, cn = n, ci = inc;
    for (int c = 0;; c += 64) {
      const unsigned long long past = __ballot(seen + ci > b);
      if (past) {
        const int f = __ffsll((long long)past) - 1;
        g = c + f;
        l = __builtin_amdgcn_readlane(cl, f) + (b - seen - __builtin_amdgcn_readlane(ci - cn, f)) * bm;
        h = __builtin_amdgcn_readlane(ch, f);
        return true;
      }
      if (c + 64 > G) return false;
      seen += __builtin_amdgcn_readlane(ci, 63);
      scan(c + 64 + lane_id(), cl, ch, cn, ci);
    }
  }
};

// First row block of group g (RowBlocks' order) and its count of blocks.
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

// W consecutive elements (VEC: one access).
template <typename ET, int W>
struct LinVec {
  typedef ET type __attribute__((ext_vector_type(W)));
};
template <typename ET, int W, bool VEC>
__device__ __forceinline__ void load_w(const ET* p, int n, float (&v)[W]) {
  if constexpr (VEC) {
    const typename LinVec<ET, W>::type t = *(const typename LinVec<ET, W>::type*)p;
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = (float)t[i];
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = i < n ? (float)p[i] : 0.f;
  }
}
template <typename ET, int W, bool VEC>
__device__ __forceinline__ void store_w(ET* p, int n, const float (&v)[W]) {
  if constexpr (VEC) {
    typename LinVec<ET, W>::type t;
#pragma unroll
    for (int i = 0; i < W; ++i) t[i] = (ET)v[i];
    *(typename LinVec<ET, W>::type*)p = t;
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (i < n) p[i] = (ET)v[i];
  }
}

// A product's output: past the caches where it exceeds them all the same
// (`stream`; uniform), so that the operands stay there.
template <typename ET, int W, bool VEC>
__device__ __forceinline__ void put_w(ET* p, int n, const float (&v)[W], int stream) {
  if constexpr (VEC) {
    if (stream) {
      typename LinVec<ET, W>::type t;
#pragma unroll
      for (int i = 0; i < W; ++i) t[i] = (ET)v[i];
      asm volatile("");  // (the compiler would make one plain store of both branches')
      __builtin_nontemporal_store(t, (typename LinVec<ET, W>::type*)p);
      asm volatile("");
      return;
    }
  }
  store_w<ET, W, VEC>(p, n, v);
}

// The epilogue of W consecutive columns c .. of R output rows m[r] (those with
// ok[r]), the columns' biases in b: z = the float32 sums + bias,
// pre-activation out, activation, residual, one rounding to the type.  VEC: a
// row's columns in one access (N % 4 == 0 and pointers that allow it), else
// one by one up to N.  The rows go through each step together, so that their
// accesses overlap.
template <typename ET, int ACT, int W, int R, bool VEC>
__device__ __forceinline__ void linear_rows(const LinearGemm& g, float (&z)[R][W], const float (&b)[W], int c,
                                            const int (&m)[R], const bool (&ok)[R]) {
  const int n = g.N - c;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < W; ++i) z[r][i] += b[i];
  if (g.pre) {
    ET* pre = static_cast<ET*>(g.pre) + c;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (ok[r]) put_w<ET, W, VEC>(pre + (long)m[r] * g.N, n, z[r], g.stream);
  }
  if constexpr (ACT == kActSwiglu) {
    constexpr int H = W / 2;
    const long No = g.N >> 1;
    float y[R][H];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < H; ++i) y[r][i] = lin_swiglu<sizeof(ET) == 2>(z[r][2 * i], z[r][2 * i + 1], g.act);
    if (g.res) {
      const ET* res = static_cast<const ET*>(g.res) + (c >> 1);
      float v[R][H];
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (ok[r]) load_w<ET, H, VEC>(res + m[r] * No, n >> 1, v[r]);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < H; ++i) y[r][i] += v[r][i];
    }
    ET* out = static_cast<ET*>(g.out) + (c >> 1);
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (ok[r]) put_w<ET, H, VEC>(out + m[r] * No, n >> 1, y[r], g.stream);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < W; ++i) z[r][i] = lin_act<sizeof(ET) == 2>(z[r][i], ACT);
    if (g.res) {
      const ET* res = static_cast<const ET*>(g.res) + c;
      float v[R][W];
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (ok[r]) load_w<ET, W, VEC>(res + (long)m[r] * g.N, n, v[r]);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < W; ++i) z[r][i] += v[r][i];
    }
    ET* out = static_cast<ET*>(g.out) + c;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (ok[r]) put_w<ET, W, VEC>(out + (long)m[r] * g.N, n, z[r], g.stream);
  }
}

// Pre-activations z + b of W consecutive columns c .. of R output rows in 8 bits:
// the lanes of one block of columns are neighbours, and every one of them is
// here (columns from N on hold zeros).
template <int W, int R>
__device__ __forceinline__ void linear_rows8(const LinearGemm& g, const float (&z)[R][W], const float (&b)[W], int c,
                                             const int (&m)[R], const bool (&ok)[R]) {
  const int n = g.N - c, bl = g.pre8.block_log;
  const int blocks = (g.N + (1 << bl) - 1) >> bl;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float v[W];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      v[i] = z[r][i] + b[i];
      top = max(top, abs_bits(v[i]));
    }
    top = lanes_max(top, bl - (W == 4 ? 2 : 1));
    const uint32_t s = r8_scale_bits(g.pre8.format, top);
    if (!ok[r] || n <= 0) continue;
    uint8_t* p = g.pre8.codes + (long)m[r] * g.N + c;
    if (g.pre8.format == R8_INT8) store_codes<R8_INT8, W>(p, n, v, r8_inverse(s));
    else store_codes<R8_E4M3, W>(p, n, v, r8_inverse(s));
    if ((c & ((1 << bl) - 1)) == 0) g.pre8.scales[(long)m[r] * blocks + (c >> bl)] = __uint_as_float(s);
  }
}

// The same of sixteen columns c .. of row m a thread, from the float32 sums of an
// output tile in LDS at `sums`, without their bias b.  A lane takes its four
// 16-byte pieces in the order i ^ swz (b lies in that order too), so that lanes
// 256 bytes apart meet different banks.
__device__ __forceinline__ void linear_codes16(const Rows8& q, int N, const char* sums, const f32x4 (&b)[4], int swz,
                                               int c, long m, bool ok, int stream) {
  f32x4 v[4];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = *(const f32x4*)(sums + ((i ^ swz) << 4)) + b[i];
#pragma unroll
    for (int k = 0; k < 4; ++k) top = max(top, abs_bits(v[i][k]));
  }
  const int bl = q.block_log;
  const uint32_t s = r8_scale_bits(q.format, lanes_max(top, bl - 4));
  const float inv = r8_inverse(s);
  u32x4 u;
  if (q.format == R8_INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = r8_encode4<R8_INT8>(v[i], inv);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = r8_encode4<R8_E4M3>(v[i], inv);
  }
  if (swz & 1) u = u32x4{u[1], u[0], u[3], u[2]};
  if (swz & 2) u = u32x4{u[2], u[3], u[0], u[1]};
  const int n = N - c;
  if (!ok || n <= 0) return;
  const auto t = __builtin_bit_cast(RowPiece<uint8_t, 16>::type, u);
  store_piece<uint8_t, 16>(q.codes + m * N + c, n, t, stream);
  if ((c & ((1 << bl) - 1)) == 0) q.scales[m * ((N + (1 << bl) - 1) >> bl) + (c >> bl)] = __uint_as_float(s);
}

// Zeros in 8 bits in the four columns from n on of row m.
__device__ __forceinline__ void linear_zero8(const Rows8& q, int N, int m, int n) {
  const int bl = q.block_log;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < N) q.codes[(long)m * N + n + i] = q.format == R8_INT8 ? 128 : 0;
  if (n < N && (n & ((1 << bl) - 1)) == 0) q.scales[(long)m * ((N + (1 << bl) - 1) >> bl) + (n >> bl)] = 1.f;
}

// f(ACT) with the activation as a compile-time constant.
template <typename F>
__host__ __device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActSwiglu: f(std::integral_constant<int, kActSwiglu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    default: f(std::integral_constant<int, kActIdentity>{});
  }
}

// Zeros in the four columns from n on of row m (behind the last group), as the
// product (MODE) would write them.
template <typename ET, int MODE>
__device__ __forceinline__ void linear_zero(const LinearGemm& g, int m, int n) {
  if constexpr (MODE != LIN_FWD) {
    const float z[4] = {};
    store_w<ET, 4, false>(static_cast<ET*>(g.out) + (long)m * g.K + n, g.K - n, z);
    return;
  }
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
