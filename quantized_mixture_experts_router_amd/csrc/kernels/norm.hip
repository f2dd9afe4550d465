// Root-mean-square norm and its gradients (norm.h).  Bound by HBM, or by launch
// latency where there are few rows: a row is read once and stays in registers
// between its sum of squares and its output.
#include <algorithm>

#include "norm.h"
#include "rows8.hpp"
#include "tokens.h"

namespace qmoe {

namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Sums of N values over a workgroup of NW wavefronts, the same bits in every
// thread; red: [2][NW][N], the caller alternates turn (one barrier a call).
template <int N, int NW>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*red)[NW][N], int turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (NW > 1) {
    if (lane_id() == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[turn][threadIdx.x >> 6][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = red[turn][0][i];
#pragma unroll
      for (int k = 1; k < NW; ++k) v[i] += red[turn][k][i];
    }
  }
}

// h of a piece: x + r in float32, rounded to the type (it is what the residual
// stream holds, so that the backward pass, which reads that, sees the same row).
template <typename ET, int W>
__device__ __forceinline__ void add_piece(typename RowPiece<ET, W>::type& x, const typename RowPiece<ET, W>::type& r) {
#pragma unroll
  for (int i = 0; i < W; ++i) x[i] = (ET)((float)x[i] + (float)r[i]);
}

// y of a piece into the outputs: rounded once to the type, and (every lane of
// the wavefront) once to 8 bits.
template <typename ET, int F, int W>
__device__ __forceinline__ void put_piece(const Norm& a, long m, int c, const float (&y)[W]) {
  const int n = a.H - c;
  if (a.y && n > 0) {
    typename RowPiece<ET, W>::type o;
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = (ET)y[i];
    store_piece<ET, W>(static_cast<ET*>(a.y) + m * a.H + c, n, o);
  }
  if constexpr (F >= 0) {
    const int bl = a.q.block_log;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) top = max(top, abs_bits(y[i]));
    const uint32_t s = r8_scale_bits<F>(lanes_max(top, bl - (W == 8 ? 3 : 2)));
    if (n > 0) {
      store_codes<F, W>(a.q.codes + m * a.H + c, n, y, r8_inverse(s));
      if ((c & ((1 << bl) - 1)) == 0) a.q.scales[m * ((a.H + (1 << bl) - 1) >> bl) + (c >> bl)] = __uint_as_float(s);
    }
  }
}

// A workgroup per row, NP pieces of 16 bytes a thread; it goes on to further
// rows with the weight in registers.
template <typename ET, int F, int NP, int TPB>
__global__ void __launch_bounds__(TPB) qmoe_rms_norm(const Norm a) {
  constexpr int W = 16 / (int)sizeof(ET), NW = TPB / 64;
  using P = typename RowPiece<ET, W>::type;
  __shared__ float red[2][NW][1];
  const int c0 = threadIdx.x * W;
  P w[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int c = c0 + j * TPB * W;
#pragma unroll
    for (int i = 0; i < W; ++i) w[j][i] = (ET)1.f;
    if (a.w) w[j] = load_piece<ET, W>(static_cast<const ET*>(a.w) + c, a.H - c);
  }
  int turn = 0;
  for (long m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
    P h[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int c = c0 + j * TPB * W;
      h[j] = load_piece<ET, W>(static_cast<const ET*>(a.x) + m * a.H + c, a.H - c);
    }
    if (a.r) {
      P r[NP];
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int c = c0 + j * TPB * W;
        r[j] = load_piece<ET, W>(static_cast<const ET*>(a.r) + m * a.H + c, a.H - c);
      }
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int c = c0 + j * TPB * W;
        add_piece<ET, W>(h[j], r[j]);
        if (a.sum) store_piece<ET, W>(static_cast<ET*>(a.sum) + m * a.H + c, a.H - c, h[j]);
      }
    }
    float ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) ss[0] = fmaf((float)h[j][i], (float)h[j][i], ss[0]);
    block_sum<1, NW>(ss, red, turn);
    const float s = 1.f / sqrtf(ss[0] / (float)a.H + a.eps);
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      float y[W];
#pragma unroll
      for (int i = 0; i < W; ++i) y[i] = (float)h[j][i] * s * (float)w[j][i];
      put_piece<ET, F, W>(a, m, c0 + j * TPB * W, y);
    }
  }
}

// Rows too long for registers: read twice.
template <typename ET, int F>
__global__ void __launch_bounds__(1024) qmoe_rms_norm_long(const Norm a) {
  constexpr int W = 16 / (int)sizeof(ET), TPB = 1024;
  using P = typename RowPiece<ET, W>::type;
  __shared__ float red[2][16][1];
  const int c0 = threadIdx.x * W;
  auto piece = [&](long m, int c) {
    P h = load_piece<ET, W>(static_cast<const ET*>(a.x) + m * a.H + c, a.H - c);
    if (a.r) add_piece<ET, W>(h, load_piece<ET, W>(static_cast<const ET*>(a.r) + m * a.H + c, a.H - c));
    return h;
  };
  int turn = 0;
  for (long m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
    float ss[1] = {0.f};
    for (int c = c0; c < a.H; c += TPB * W) {
      const P h = piece(m, c);
      if (a.sum && a.r) store_piece<ET, W>(static_cast<ET*>(a.sum) + m * a.H + c, a.H - c, h);
#pragma unroll
      for (int i = 0; i < W; ++i) ss[0] = fmaf((float)h[i], (float)h[i], ss[0]);
    }
    block_sum<1, 16>(ss, red, turn);
    const float s = 1.f / sqrtf(ss[0] / (float)a.H + a.eps);
    // (every lane of a wavefront takes part in its blocks' largest magnitude)
    for (int base = 0; base < a.H; base += TPB * W) {
      const int c = base + c0;
      float y[W] = {};
      if (c < a.H) {
        const P h = piece(m, c);
        P w;
        if (a.w) w = load_piece<ET, W>(static_cast<const ET*>(a.w) + c, a.H - c);
#pragma unroll
        for (int i = 0; i < W; ++i) y[i] = (float)h[i] * s * (a.w ? (float)w[i] : 1.f);
      }
      put_piece<ET, F, W>(a, m, c, y);
    }
  }
}

// A workgroup per row at a time; the weight's gradient of its rows stays in
// registers and leaves as one row of partial sums.
template <typename ET, int NP, int TPB>
__global__ void __launch_bounds__(TPB) qmoe_rms_norm_grad(const NormGrad a, long ldp) {
  constexpr int W = 16 / (int)sizeof(ET), NW = TPB / 64;
  using P = typename RowPiece<ET, W>::type;
  __shared__ float red[2][NW][2];
  const int c0 = threadIdx.x * W;
  P w[NP];
  float acc[NP][W];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int c = c0 + j * TPB * W;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      w[j][i] = (ET)1.f;
      acc[j][i] = 0.f;
    }
    if (a.w) w[j] = load_piece<ET, W>(static_cast<const ET*>(a.w) + c, a.H - c);
  }
  int turn = 0;
  for (long m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
    P h[NP], g[NP], d[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int c = c0 + j * TPB * W;
      h[j] = load_piece<ET, W>(static_cast<const ET*>(a.h) + m * a.H + c, a.H - c);
      g[j] = load_piece<ET, W>(static_cast<const ET*>(a.dy) + m * a.H + c, a.H - c);
      d[j] = P{};
      if (a.ds && a.dh) d[j] = load_piece<ET, W>(static_cast<const ET*>(a.ds) + m * a.H + c, a.H - c);
    }
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        v[0] = fmaf((float)h[j][i], (float)h[j][i], v[0]);
        v[1] = fmaf((float)g[j][i] * (float)w[j][i], (float)h[j][i], v[1]);
      }
    block_sum<2, NW>(v, red, turn);
    const float s = 1.f / sqrtf(v[0] / (float)a.H + a.eps), mean = v[1] * s / (float)a.H;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int c = c0 + j * TPB * W;
      P o;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float n = (float)h[j][i] * s, gi = (float)g[j][i];
        o[i] = (ET)fmaf(s, gi * (float)w[j][i] - n * mean, (float)d[j][i]);
        acc[j][i] = fmaf(gi, n, acc[j][i]);
      }
      if (a.dh) store_piece<ET, W>(static_cast<ET*>(a.dh) + m * a.H + c, a.H - c, o);
    }
  }
  if (!a.dw) return;
#pragma unroll
  for (int j = 0; j < NP; ++j)
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const int c = c0 + j * TPB * W + i;
      if (c < ldp) *(f32x4*)(a.partial + blockIdx.x * ldp + c) = f32x4{acc[j][i], acc[j][i + 1], acc[j][i + 2], acc[j][i + 3]};
    }
}

// Rows too long for registers: read twice; 1 / root mean square of every row
// into rstd for the weight's gradient.
template <typename ET>
__global__ void __launch_bounds__(1024) qmoe_rms_norm_grad_long(const NormGrad a, float* __restrict__ rstd) {
  constexpr int W = 16 / (int)sizeof(ET), TPB = 1024;
  using P = typename RowPiece<ET, W>::type;
  __shared__ float red[2][16][2];
  const ET* w = static_cast<const ET*>(a.w);
  int turn = 0;
  for (long m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
    const ET* hp = static_cast<const ET*>(a.h) + m * a.H;
    const ET* gp = static_cast<const ET*>(a.dy) + m * a.H;
    float v[2] = {0.f, 0.f};
    for (int c = threadIdx.x * W; c < a.H; c += TPB * W) {
      const P h = load_piece<ET, W>(hp + c, a.H - c), g = load_piece<ET, W>(gp + c, a.H - c);
      P wp;
      if (w) wp = load_piece<ET, W>(w + c, a.H - c);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        v[0] = fmaf((float)h[i], (float)h[i], v[0]);
        v[1] = fmaf((float)g[i] * (w ? (float)wp[i] : 1.f), (float)h[i], v[1]);
      }
    }
    block_sum<2, 16>(v, red, turn);
    const float s = 1.f / sqrtf(v[0] / (float)a.H + a.eps), mean = v[1] * s / (float)a.H;
    if (a.dw && threadIdx.x == 0) rstd[m] = s;
    if (!a.dh) continue;
    for (int c = threadIdx.x * W; c < a.H; c += TPB * W) {
      const int n = a.H - c;
      const P h = load_piece<ET, W>(hp + c, n), g = load_piece<ET, W>(gp + c, n);
      P wp, d = {}, o;
      if (w) wp = load_piece<ET, W>(w + c, n);
      if (a.ds) d = load_piece<ET, W>(static_cast<const ET*>(a.ds) + m * a.H + c, n);
#pragma unroll
      for (int i = 0; i < W; ++i)
        o[i] = (ET)fmaf(s, (float)g[i] * (w ? (float)wp[i] : 1.f) - (float)h[i] * s * mean, (float)d[i]);
      store_piece<ET, W>(static_cast<ET*>(a.dh) + m * a.H + c, n, o);
    }
  }
}

// Partial sums of the weight's gradient from rstd: workgroup (x, y) takes the
// columns of x and the rows y, y + gridDim.y, ...
template <typename ET>
__global__ void __launch_bounds__(256) qmoe_norm_weight_grad(const NormGrad a, const float* __restrict__ rstd,
                                                             float* __restrict__ partial, long ldp) {
  constexpr int W = 16 / (int)sizeof(ET);
  const int c = (blockIdx.x * 256 + threadIdx.x) * W, n = a.H - c;
  if (n <= 0) return;
  float acc[W] = {};
  for (long m = blockIdx.y; m < a.M; m += gridDim.y) {
    const auto h = load_piece<ET, W>(static_cast<const ET*>(a.h) + m * a.H + c, n);
    const auto g = load_piece<ET, W>(static_cast<const ET*>(a.dy) + m * a.H + c, n);
    const float s = rstd[m];
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = fmaf((float)g[i], (float)h[i] * s, acc[i]);
  }
#pragma unroll
  for (int i = 0; i < W; i += 4)
    if (c + i < ldp) *(f32x4*)(partial + blockIdx.y * ldp + c + i) = f32x4{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
}

// dw = sum of B rows of partial sums: 64 columns a workgroup, four a thread,
// sixteen threads over the rows of each (in a fixed order).
template <typename ET>
__global__ void __launch_bounds__(256) qmoe_norm_sum(const float* __restrict__ partial, long ldp, int B, int H,
                                                     ET* __restrict__ dw) {
  __shared__ f32x4 red[16][16];
  const int q = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int c = (blockIdx.x * 16 + q) * 4;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c < ldp) {
#pragma unroll 8
    for (int b = g; b < B; b += 16) s += *(const f32x4*)(partial + b * ldp + c);
  }
  red[g][q] = s;
  __syncthreads();
  if (g > 0) return;
#pragma unroll
  for (int k = 1; k < 16; ++k) s += red[k][q];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c + i < H) dw[c + i] = (ET)s[i];
}

constexpr int kCUs = 256;
constexpr int kLongRows = 256;  // rows of partial sums for rows too long for registers

// Threads a row and pieces a thread; 0 pieces: too long for registers.
struct NormShape {
  int threads, np;
};
NormShape norm_shape(long pieces) {
  if (pieces <= 64) return {64, 1};
  if (pieces <= 128) return {64, 2};
  if (pieces <= 256) return {256, 1};
  if (pieces <= 512) return {256, 2};
  if (pieces <= 1024) return {256, 4};
  if (pieces <= 2048) return {1024, 2};
  if (pieces <= 4096) return {1024, 4};
  return {1024, 0};
}
unsigned norm_grid(long M, int threads) { return (unsigned)std::min<long>(M, kCUs * (2048 / threads)); }
// (fewer in the backward pass: each leaves a row of partial sums)
unsigned norm_grad_grid(long M, int threads) { return (unsigned)std::min<long>(M, kCUs * std::max(1, 512 / threads)); }

// f(TPB, NP) with both as compile-time constants.
template <typename G>
void with_shape(const NormShape& s, G f) {
#define QMOE_SHAPE(T, N) \
  if (s.threads == T && s.np == N) return f(std::integral_constant<int, T>{}, std::integral_constant<int, N>{});
  QMOE_SHAPE(64, 1)
  QMOE_SHAPE(64, 2)
  QMOE_SHAPE(256, 1)
  QMOE_SHAPE(256, 2)
  QMOE_SHAPE(256, 4)
  QMOE_SHAPE(1024, 2)
  QMOE_SHAPE(1024, 4)
#undef QMOE_SHAPE
}

template <typename ET, int F>
hipError_t norm_t(const Norm& a, hipStream_t st) {
  constexpr int W = 16 / (int)sizeof(ET);
  const NormShape s = norm_shape((a.H + W - 1) / W);
  const dim3 grid(norm_grid(a.M, s.threads)), block(s.threads);
  if (s.np == 0) {
    hipLaunchKernelGGL((qmoe_rms_norm_long<ET, F>), grid, block, 0, st, a);
  } else {
    with_shape(s, [&](auto t, auto n) {
      hipLaunchKernelGGL((qmoe_rms_norm<ET, F, decltype(n)::value, decltype(t)::value>), grid, block, 0, st, a);
    });
  }
  return hipGetLastError();
}

template <typename ET>
hipError_t norm_format(const Norm& a, hipStream_t st) {
  if (!a.q.codes) return norm_t<ET, -1>(a, st);
  if (a.q.format == R8_INT8) return norm_t<ET, R8_INT8>(a, st);
  return norm_t<ET, R8_E4M3>(a, st);
}

long padded(long H) { return (H + 3) / 4 * 4; }

template <typename ET>
hipError_t norm_grad_t(const NormGrad& a, hipStream_t st) {
  constexpr int W = 16 / (int)sizeof(ET);
  const NormShape s = norm_shape((a.H + W - 1) / W);
  const long ldp = padded(a.H);
  const float* partial = a.partial;
  unsigned rows = 0;
  if (a.M > 0) {
    rows = norm_grad_grid(a.M, s.threads);
    if (s.np == 0) {
      float* rstd = a.partial + kLongRows * ldp;
      hipLaunchKernelGGL(qmoe_rms_norm_grad_long<ET>, dim3(rows), dim3(1024), 0, st, a, rstd);
      rows = (unsigned)std::min<long>(a.M, kLongRows);
      if (a.dw)
        hipLaunchKernelGGL(qmoe_norm_weight_grad<ET>, dim3((unsigned)((a.H + 256 * W - 1) / (256 * W)), rows), dim3(256), 0, st, a, rstd, a.partial, ldp);
    } else {
      with_shape(s, [&](auto t, auto n) {
        hipLaunchKernelGGL((qmoe_rms_norm_grad<ET, decltype(n)::value, decltype(t)::value>), dim3(rows), dim3(s.threads), 0, st, a, ldp);
      });
    }
  }
  if (a.dw) hipLaunchKernelGGL(qmoe_norm_sum<ET>, dim3((unsigned)((a.H + 63) / 64)), dim3(256), 0, st, partial, ldp, (int)rows, a.H, (ET*)a.dw);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(int type, const Norm& a, hipStream_t st) {
  if (type == ROW_F32) return norm_format<float>(a, st);
  if (type == ROW_F16) return norm_format<_Float16>(a, st);
  return norm_format<__bf16>(a, st);
}

size_t norm_partials(int type, long M, long H) {
  if (M == 0) return 0;
  const long W = type == ROW_F32 ? 4 : 8;
  const NormShape s = norm_shape((H + W - 1) / W);
  if (s.np == 0) return (size_t)(kLongRows * padded(H) + M);
  return (size_t)norm_grad_grid(M, s.threads) * (size_t)padded(H);
}

hipError_t launch_rms_norm_grad(int type, const NormGrad& a, hipStream_t st) {
  if (type == ROW_F32) return norm_grad_t<float>(a, st);
  if (type == ROW_F16) return norm_grad_t<_Float16>(a, st);
  return norm_grad_t<__bf16>(a, st);
}

}  // namespace qmoe
