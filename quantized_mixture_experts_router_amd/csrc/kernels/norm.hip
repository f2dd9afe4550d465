// Root-mean-square norm and its gradients (norm.h).  Bound by HBM, or by launch
// latency where there are few rows: a row is read once and stays in registers
// between its sum of squares and its output.
#include <algorithm>

#include "launches.h"
#include "norm.h"
#include "rows8.hpp"
#include "tokens.h"

namespace qmoe {

namespace {

// Sum over the TPR lanes (8, 16, 32 or 64) of a row.
template <int TPR>
__device__ __forceinline__ float lanes_sum(float v) {
  auto add = [](float x, uint32_t y) { return x + __uint_as_float(y); };
  v = add(v, dpp_from<kDppXor1>(__float_as_uint(v)));
  v = add(v, dpp_from<kDppXor2>(__float_as_uint(v)));
  v = add(v, dpp_from<kDppHalf>(__float_as_uint(v)));
  if constexpr (TPR > 8) v = add(v, dpp_from<kDppRow>(__float_as_uint(v)));
  if constexpr (TPR > 16) {
    uint32_t x = __float_as_uint(v), y = x;
    swap16(x, y);
    v = add(__uint_as_float(x), y);
  }
  if constexpr (TPR > 32) {
    uint32_t x = __float_as_uint(v), y = x;
    swap32(x, y);
    v = add(__uint_as_float(x), y);
  }
  return v;
}

// Rows of a workgroup that gives TPR threads to each: 256 threads, or one row.
constexpr int rows_of(int TPR) { return TPR < 256 ? 256 / TPR : 1; }
constexpr int threads_of(int TPR) { return TPR < 256 ? 256 : TPR; }

// Sums of N values over the TPR threads of a row, the same bits in every one;
// red: [2][wavefronts][N] for rows of several wavefronts, where the caller
// alternates turn (one barrier a call).
template <typename S, int N, int TPR>
__device__ __forceinline__ void row_sum(S (&v)[N], S (*red)[threads_of(TPR) / 64][N], int turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (std::is_same<S, double>::value) v[i] = wave_sum_double<TPR < 64 ? TPR : 64>(v[i]);
    else v[i] = lanes_sum<TPR < 64 ? TPR : 64>(v[i]);
  }
  if constexpr (TPR > 64) {
    if (lane_id() == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[turn][threadIdx.x >> 6][i] = v[i];
    }
    __syncthreads();
    const int first = threadIdx.x / TPR * (TPR / 64);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = red[turn][first][i];
#pragma unroll
      for (int k = 1; k < TPR / 64; ++k) v[i] += red[turn][first + k][i];
    }
  }
}

// 1 / sqrt(ss / H + eps) as the sum of two floats.  A value goes to 8 bits by
// the side of a border that it lies on, and each float32 rounding before puts a
// few in a million on the other: the threads' float32 sums are added in 64 bits, s
// keeps its tail, and h s w is rounded once (forward only; next to HBM this is
// free).  Squares that pass float32 leave 0.
struct RowScale {
  float hi, lo;
};
__device__ __forceinline__ RowScale row_scale(double ss, int H, float eps) {
  const double x = ss / (double)H + (double)eps;
  // the hardware's estimate (2^-22 at least) and a step of Newton's method
  double y = __builtin_amdgcn_rsq(x);
  y = fma(y * 0.5, fma(-x * y, y, 1.0), y);
  y = x > 1e300 ? 0.0 : y;
  const float hi = (float)y;
  return {hi, (float)(y - (double)hi)};
}
// h s w.  h s first: it is at most sqrt(H), while h w may pass float32's range where the result does not.
__device__ __forceinline__ float scaled(float h, float w, const RowScale& s) {
  const float n = h * s.hi;
  const float low = fmaf(h, s.lo, fmaf(h, s.hi, -n));
  return fmaf(n, w, low * w);
}

// h of a piece: x + r in float32, rounded to the type (it is what the residual
// stream holds, so that the backward pass, which reads that, sees the same row).
template <typename ET, int W>
__device__ __forceinline__ void add_piece(typename RowPiece<ET, W>::type& x, const typename RowPiece<ET, W>::type& r) {
#pragma unroll
  for (int i = 0; i < W; ++i) x[i] = (ET)((float)x[i] + (float)r[i]);
}

// y of a piece into the outputs: rounded once to the type, and (every lane of a
// row of 2^lanes lanes) once to 8 bits.
template <typename ET, int F, int W>
__device__ __forceinline__ void put_piece(const Norm& a, long m, int c, const float (&y)[W], int lanes = 6) {
  const int n = m < a.M ? a.H - c : 0;
  if (a.y && n > 0) {
    typename RowPiece<ET, W>::type o;
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = (ET)y[i];
    store_piece<ET, W>(static_cast<ET*>(a.y) + m * a.H + c, n, o, a.stream);
  }
  if constexpr (F >= 0) {
    const int bl = a.q.block_log;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) top = max(top, abs_bits(y[i]));
    const uint32_t s = r8_scale_bits<F>(lanes_max(top, min(bl - (W == 8 ? 3 : 2), lanes)));
    if (n > 0) {
      store_codes<F, W>(a.q.codes + m * a.H + c, n, y, r8_inverse(s));
      if ((c & ((1 << bl) - 1)) == 0) a.q.scales[m * ((a.H + (1 << bl) - 1) >> bl) + (c >> bl)] = __uint_as_float(s);
    }
  }
}

// TPR threads a row, NP pieces of 16 bytes each; a workgroup of 256 threads or
// more takes a row, or several, and goes on to further ones with the weight in
// registers.  Bfloat16 with residual: 8192 x 4096 48 us for 268 MB (5.6 TB/s), with
// 8 bits beside it 53 to 55 us for 303 MB; 65536 x 64 8.5 us (a wavefront a row: 20 us).
template <typename ET, int F, int NP, int TPR>
__global__ void __launch_bounds__(threads_of(TPR)) qmoe_rms_norm(const Norm a) {
  constexpr int W = 16 / (int)sizeof(ET), R = rows_of(TPR);
  constexpr int kLanes = TPR >= 64 ? 6 : TPR == 32 ? 5 : TPR == 16 ? 4 : 3;
  using P = typename RowPiece<ET, W>::type;
  __shared__ double red[2][threads_of(TPR) / 64][1];
  const int c0 = threadIdx.x % TPR * W;
  P w[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int c = c0 + j * TPR * W;
#pragma unroll
    for (int i = 0; i < W; ++i) w[j][i] = (ET)1.f;
    if (a.w) w[j] = load_piece<ET, W>(static_cast<const ET*>(a.w) + c, a.H - c);
  }
  int turn = 0;
  for (long m0 = (long)blockIdx.x * R; m0 < a.M; m0 += (long)gridDim.x * R, turn ^= 1) {
    const long m = m0 + threadIdx.x / TPR;
    const int H = m < a.M ? a.H : 0;
    P h[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int c = c0 + j * TPR * W;
      h[j] = load_piece<ET, W>(static_cast<const ET*>(a.x) + m * a.H + c, H - c);
    }
    if (a.r) {
      P r[NP];
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int c = c0 + j * TPR * W;
        r[j] = load_piece<ET, W>(static_cast<const ET*>(a.r) + m * a.H + c, H - c);
      }
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int c = c0 + j * TPR * W;
        add_piece<ET, W>(h[j], r[j]);
        if (a.sum) store_piece<ET, W>(static_cast<ET*>(a.sum) + m * a.H + c, H - c, h[j], a.stream);
      }
    }
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) sq = fmaf((float)h[j][i], (float)h[j][i], sq);
    double ss[1] = {sq};
    row_sum<double, 1, TPR>(ss, red, turn);
    const RowScale s = row_scale(ss[0], a.H, a.eps);
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      float y[W];
#pragma unroll
      for (int i = 0; i < W; ++i) y[i] = scaled((float)h[j][i], (float)w[j][i], s);
      put_piece<ET, F, W>(a, m, c0 + j * TPR * W, y, kLanes);
    }
  }
}

// Rows too long for registers: read twice.  512 x 40000 bfloat16: 38 us for 164 MB.
template <typename ET, int F>
__global__ void __launch_bounds__(1024) qmoe_rms_norm_long(const Norm a) {
  constexpr int W = 16 / (int)sizeof(ET), TPR = 1024;
  using P = typename RowPiece<ET, W>::type;
  __shared__ double red[2][16][1];
  const int c0 = threadIdx.x * W;
  auto piece = [&](long m, int c) {
    P h = load_piece<ET, W>(static_cast<const ET*>(a.x) + m * a.H + c, a.H - c);
    if (a.r) add_piece<ET, W>(h, load_piece<ET, W>(static_cast<const ET*>(a.r) + m * a.H + c, a.H - c));
    return h;
  };
  int turn = 0;
  for (long m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
    double ss[1] = {0.0};
    for (int c = c0; c < a.H; c += TPR * W) {
      const P h = piece(m, c);
      if (a.sum && a.r) store_piece<ET, W>(static_cast<ET*>(a.sum) + m * a.H + c, a.H - c, h, a.stream);
      float sq = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) sq = fmaf((float)h[i], (float)h[i], sq);
      ss[0] += (double)sq;
    }
    row_sum<double, 1, TPR>(ss, red, turn);
    const RowScale s = row_scale(ss[0], a.H, a.eps);
    // (every lane of a wavefront takes part in its blocks' largest magnitude)
    for (int base = 0; base < a.H; base += TPR * W) {
      const int c = base + c0;
      float y[W] = {};
      if (c < a.H) {
        const P h = piece(m, c);
        P w;
        if (a.w) w = load_piece<ET, W>(static_cast<const ET*>(a.w) + c, a.H - c);
#pragma unroll
        for (int i = 0; i < W; ++i) y[i] = scaled((float)h[i], a.w ? (float)w[i] : 1.f, s);
      }
      put_piece<ET, F, W>(a, m, c, y);
    }
  }
}

// 8192 x 4096 bfloat16 with a gradient at the sum: 50 to 51 us for 268 MB and the
// partial sums, 5.4 TB/s (inputs in part still in the last level of cache), 65536 x
// 64 8.8 us; float32 8192 x 4096 93 us for 537 MB.
// Threads and rows as above; the weight's gradient of a workgroup's rows stays
// in registers and leaves as one row of partial sums.
template <typename ET, int NP, int TPR>
__global__ void __launch_bounds__(threads_of(TPR)) qmoe_rms_norm_grad(const NormGrad a, long ldp) {
  constexpr int W = 16 / (int)sizeof(ET), R = rows_of(TPR);
  using P = typename RowPiece<ET, W>::type;
  __shared__ float red[2][threads_of(TPR) / 64][2];
  const int c0 = threadIdx.x % TPR * W;
  P w[NP];
  float acc[NP][W];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int c = c0 + j * TPR * W;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      w[j][i] = (ET)1.f;
      acc[j][i] = 0.f;
    }
    if (a.w) w[j] = load_piece<ET, W>(static_cast<const ET*>(a.w) + c, a.H - c);
  }
  int turn = 0;
  for (long m0 = (long)blockIdx.x * R; m0 < a.M; m0 += (long)gridDim.x * R, turn ^= 1) {
    const long m = m0 + threadIdx.x / TPR;
    const int H = m < a.M ? a.H : 0;
    P h[NP], g[NP], d[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int c = c0 + j * TPR * W;
      h[j] = load_piece<ET, W>(static_cast<const ET*>(a.h) + m * a.H + c, H - c);
      g[j] = load_piece<ET, W>(static_cast<const ET*>(a.dy) + m * a.H + c, H - c);
      d[j] = P{};
      if (a.ds && a.dh) d[j] = load_piece<ET, W>(static_cast<const ET*>(a.ds) + m * a.H + c, H - c);
    }
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        v[0] = fmaf((float)h[j][i], (float)h[j][i], v[0]);
        v[1] = fmaf((float)g[j][i] * (float)w[j][i], (float)h[j][i], v[1]);
      }
    row_sum<float, 2, TPR>(v, red, turn);
    const float s = 1.f / sqrtf(v[0] / (float)a.H + a.eps), mean = v[1] * s / (float)a.H;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int c = c0 + j * TPR * W;
      P o;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float n = (float)h[j][i] * s, gi = (float)g[j][i];
        o[i] = (ET)fmaf(s, gi * (float)w[j][i] - n * mean, (float)d[j][i]);
        acc[j][i] = fmaf(gi, n, acc[j][i]);
      }
      if (a.dh) store_piece<ET, W>(static_cast<ET*>(a.dh) + m * a.H + c, H - c, o, a.stream);
    }
  }
  if (!a.dw) return;
  if constexpr (R > 1) {
    // a column's sums of the workgroup's R rows at a time, in their order
    __shared__ float cols[R][TPR * W];
#pragma unroll
    for (int i = 0; i < W; ++i) cols[threadIdx.x / TPR][c0 + i] = acc[0][i];
    __syncthreads();
    for (int c = threadIdx.x; c < TPR * W && c < ldp; c += 256) {
      float s = 0.f;
#pragma unroll 8
      for (int r = 0; r < R; ++r) s += cols[r][c];
      a.partial[blockIdx.x * ldp + c] = s;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NP; ++j)
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const int c = c0 + j * TPR * W + i;
      if (c < ldp) *(f32x4*)(a.partial + blockIdx.x * ldp + c) = f32x4{acc[j][i], acc[j][i + 1], acc[j][i + 2], acc[j][i + 3]};
    }
}

// Rows too long for registers: read twice; 1 / root mean square of every row
// into rstd for the weight's gradient, which reads them again.  1024 x 32768
// bfloat16: 63 us for 268 MB, and 27 for the weight's gradient.
template <typename ET>
__global__ void __launch_bounds__(1024) qmoe_rms_norm_grad_long(const NormGrad a, float* __restrict__ rstd) {
  constexpr int W = 16 / (int)sizeof(ET), TPR = 1024;
  using P = typename RowPiece<ET, W>::type;
  __shared__ float red[2][16][2];
  const ET* w = static_cast<const ET*>(a.w);
  int turn = 0;
  for (long m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
    const ET* hp = static_cast<const ET*>(a.h) + m * a.H;
    const ET* gp = static_cast<const ET*>(a.dy) + m * a.H;
    float v[2] = {0.f, 0.f};
    for (int c = threadIdx.x * W; c < a.H; c += TPR * W) {
      const P h = load_piece<ET, W>(hp + c, a.H - c), g = load_piece<ET, W>(gp + c, a.H - c);
      P wp;
      if (w) wp = load_piece<ET, W>(w + c, a.H - c);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        v[0] = fmaf((float)h[i], (float)h[i], v[0]);
        v[1] = fmaf((float)g[i] * (w ? (float)wp[i] : 1.f), (float)h[i], v[1]);
      }
    }
    row_sum<float, 2, TPR>(v, red, turn);
    const float s = 1.f / sqrtf(v[0] / (float)a.H + a.eps), mean = v[1] * s / (float)a.H;
    if (a.dw && threadIdx.x == 0) rstd[m] = s;
    if (!a.dh) continue;
    for (int c = threadIdx.x * W; c < a.H; c += TPR * W) {
      const int n = a.H - c;
      const P h = load_piece<ET, W>(hp + c, n), g = load_piece<ET, W>(gp + c, n);
      P wp, d = {}, o;
      if (w) wp = load_piece<ET, W>(w + c, n);
      if (a.ds) d = load_piece<ET, W>(static_cast<const ET*>(a.ds) + m * a.H + c, n);
#pragma unroll
      for (int i = 0; i < W; ++i)
        o[i] = (ET)fmaf(s, (float)g[i] * (w ? (float)wp[i] : 1.f) - (float)h[i] * s * mean, (float)d[i]);
      store_piece<ET, W>(static_cast<ET*>(a.dh) + m * a.H + c, n, o, a.stream);
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

// dw = sum of B rows of partial sums: 32 columns a workgroup, four a thread,
// thirty-two threads over the rows of each (in a fixed order).
template <typename ET>
__global__ void __launch_bounds__(256) qmoe_norm_sum(const float* __restrict__ partial, long ldp, int B, int H,
                                                     ET* __restrict__ dw) {
  __shared__ f32x4 red[32][8];
  const int q = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int c = (blockIdx.x * 8 + q) * 4;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c < ldp) {
#pragma unroll 8
    for (int b = g; b < B; b += 32) s += *(const f32x4*)(partial + b * ldp + c);
  }
  red[g][q] = s;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int k = threadIdx.x;  // a column a thread
  float t = 0.f;
#pragma unroll
  for (int r = 0; r < 32; ++r) t += red[r][k >> 2][k & 3];
  if (blockIdx.x * 32 + k < H) dw[blockIdx.x * 32 + k] = (ET)t;
}

constexpr int kCUs = 256;
constexpr int kLongRows = 256;  // rows of partial sums for rows too long for registers

// Threads a row and pieces a thread; 0 pieces: too long for registers.
// Few rows: a piece a thread, up to 1024 (16 x 4096 bfloat16 2.9 and with 8 bits 3.4
// us, with 256 x 2 3.2 and 3.9, with 64 x 8 5.6 and 7.9); many: 256 threads where
// the row allows (8192 x 4096 48 and 57 us, 128 x 4 48 and 60, 1024 x 1 49 and 72).
// (512 x 8 in float32 spills 17 registers in the backward pass: 2048 x 16384 104 us for 537 MB.)
struct NormShape {
  int threads, np;
};
NormShape norm_shape(long M, long pieces, long most) {
  if (pieces <= 8) return {8, 1};
  if (pieces <= 16) return {16, 1};
  if (pieces <= 32) return {32, 1};
  if (pieces <= 64) return {64, 1};
  if (pieces <= 128) return {128, 1};
  if (pieces <= 256) return {256, 1};
  if (M <= 2 * kCUs && pieces <= 512) return {512, 1};
  if (M <= 2 * kCUs && pieces <= 1024) return {1024, 1};
  if (pieces <= 512) return {256, 2};
  if (pieces <= 1024) return {256, 4};
  if (pieces <= 2048) return {512, 4};
  if (pieces <= most) return {512, 8};
  return {1024, 0};
}
unsigned norm_grid(long M, const NormShape& s) {
  const long rows = rows_of(s.threads);
  return (unsigned)std::min<long>((M + rows - 1) / rows, kCUs * (2048 / threads_of(s.threads)));
}
// Fewer in the backward pass, each of which leaves a row of partial sums.  us with
// their sum, on 1 / 2 / 4 / 8 workgroups a compute unit, bfloat16: 8192 x 8192 (256 x 4)
// 115 / 102 / 106 / 117, 8192 x 4096 (256 x 2) 67 / 57 / 57 / 61, 8192 x 2048 (256 x 1)
// 50 / 34 / 32 / 35, 8192 x 1024 (128 x 1) 25 / 20 / 18 / 22, 65536 x 64 (8 x 1) 13 / 11 /
// 11 / 13; float32 8192 x 4096 (256 x 4) 100 / 98 / 101 / 104.  On 1 / 2 / 4: bfloat16
// 4096 x 16384 (512 x 4) 109 / 115 / 127, 512 x 8192 (1024 x 1) 14 / 17 / 18, float32
// 2048 x 16384 (512 x 8) 108 / 110 / 120.
unsigned norm_grad_grid(long M, const NormShape& s) {
  const long rows = rows_of(s.threads);
  const long per = s.threads <= 256 && s.np == 1 ? 4 : s.threads <= 256 ? 2 : 1;
  return (unsigned)std::min<long>((M + rows - 1) / rows, kCUs * per);
}
// The longest rows (in pieces) that stay in registers: in the backward pass 16-bit
// rows of 512 threads x 8 pieces would spill 900 bytes a lane (1024 x 32768: 254 us).
template <typename ET>
constexpr long kMostGrad = sizeof(ET) == 4 ? 4096 : 2048;

// f(TPR, NP) with both as compile-time constants.
template <typename G>
void with_shape(const NormShape& s, G f) {
#define QMOE_SHAPE(T, N) \
  if (s.threads == T && s.np == N) return f(std::integral_constant<int, T>{}, std::integral_constant<int, N>{});
  QMOE_SHAPE(8, 1)
  QMOE_SHAPE(16, 1)
  QMOE_SHAPE(32, 1)
  QMOE_SHAPE(64, 1)
  QMOE_SHAPE(128, 1)
  QMOE_SHAPE(256, 1)
  QMOE_SHAPE(512, 1)
  QMOE_SHAPE(1024, 1)
  QMOE_SHAPE(256, 2)
  QMOE_SHAPE(256, 4)
  QMOE_SHAPE(512, 4)
  QMOE_SHAPE(512, 8)
#undef QMOE_SHAPE
}

template <typename ET, int F>
hipError_t norm_t(Norm a, hipStream_t st) {
  constexpr int W = 16 / (int)sizeof(ET);
  a.stream = a.M * a.H * (long)((a.y ? sizeof(ET) : 0) + (a.sum ? sizeof(ET) : 0) + (F >= 0 ? 1 : 0)) >= kStreamBytes;
  const NormShape s = norm_shape(a.M, (a.H + W - 1) / W, 4096);
  const dim3 grid(norm_grid(a.M, s)), block(threads_of(s.threads));
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
hipError_t norm_grad_t(NormGrad a, hipStream_t st) {
  constexpr int W = 16 / (int)sizeof(ET);
  a.stream = a.dh && a.M * a.H * (long)sizeof(ET) >= kStreamBytes;
  const NormShape s = norm_shape(a.M, (a.H + W - 1) / W, kMostGrad<ET>);
  const long ldp = padded(a.H);
  const float* partial = a.partial;
  unsigned rows = 0;
  if (a.M > 0) {
    rows = norm_grad_grid(a.M, s);
    if (s.np == 0) {
      float* rstd = a.partial + kLongRows * ldp;
      hipLaunchKernelGGL(qmoe_rms_norm_grad_long<ET>, dim3(rows), dim3(1024), 0, st, a, rstd);
      rows = (unsigned)std::min<long>(a.M, kLongRows);
      if (a.dw)
        hipLaunchKernelGGL(qmoe_norm_weight_grad<ET>, dim3((unsigned)((a.H + 256 * W - 1) / (256 * W)), rows), dim3(256), 0, st, a, rstd, a.partial, ldp);
    } else {
      with_shape(s, [&](auto t, auto n) {
        constexpr int T = decltype(t)::value, N = decltype(n)::value;
        if constexpr (T * N <= kMostGrad<ET>)
          hipLaunchKernelGGL((qmoe_rms_norm_grad<ET, N, T>), dim3(rows), dim3(threads_of(s.threads)), 0, st, a, ldp);
      });
    }
  }
  if (a.dw) hipLaunchKernelGGL(qmoe_norm_sum<ET>, dim3((unsigned)((a.H + 31) / 32)), dim3(256), 0, st, partial, ldp, (int)rows, a.H, (ET*)a.dw);
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
  const NormShape s = norm_shape(M, (H + W - 1) / W, type == ROW_F32 ? kMostGrad<float> : kMostGrad<_Float16>);
  if (s.np == 0) return (size_t)(kLongRows * padded(H) + M);
  return (size_t)norm_grad_grid(M, s) * (size_t)padded(H);
}

hipError_t launch_rms_norm_grad(int type, const NormGrad& a, hipStream_t st) {
  if (type == ROW_F32) return norm_grad_t<float>(a, st);
  if (type == ROW_F16) return norm_grad_t<_Float16>(a, st);
  return norm_grad_t<__bf16>(a, st);
}

}  // namespace qmoe
