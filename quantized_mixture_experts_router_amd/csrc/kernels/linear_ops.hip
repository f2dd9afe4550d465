// The linear layers' passes beside the matrix kernel (linear.h): the sum of
// split reductions with the epilogue, the activation's gradient with column
// sums, the bias gradient and row padding.  All are bound by HBM.
#include <algorithm>

#include "launches.h"
#include "linear_common.hpp"

namespace qmoe {

namespace {

// Group of output row m (rows behind the last group: G): binary search for
// the first group whose end lies past m; offsets as group_rows takes them.
__device__ __forceinline__ int group_of_row(const int* __restrict__ offsets, int G, int M, int m) {
  if (!offsets) return 0;
  int a = 0, b = G;
  while (a < b) {
    const int c = (a + b) >> 1;
    int lo, hi;
    group_rows(offsets, G, M, c, lo, hi);
    if (hi > m) b = c;
    else a = c + 1;
  }
  return a;
}

// Four columns of one output row a thread (two where rows allow no wide
// access): the ranges' sums added in range order, then the epilogue (or the
// store).  1001 x 1411 float32, two ranges, gelu, pre-activations kept: 8.2 us for
// 23 MB (four columns a thread, whose single stores then lie 16 bytes apart, took
// 2.6 us more).
template <typename ET, int MODE, bool VEC>
__global__ void __launch_bounds__(256) qmoe_linear_finish(const LinearGemm g) {
  constexpr int W = VEC ? 4 : 2;
  typedef float V __attribute__((ext_vector_type(W)));
  const int cols = MODE == LIN_FWD ? g.N : g.K;
  const long ldp = (cols + 3) & ~3;
  const long rows = MODE == LIN_DW ? (long)g.G * g.N : g.M;
  // (fewer than 2^31 outputs where a reduction is split)
  const uint32_t i = blockIdx.x * 256 + threadIdx.x, per = (uint32_t)ldp / W;
  const long row = i / per;
  const int c = (int)(i - (uint32_t)row * per) * W;
  if (row >= rows) return;
  int grp = 0;
  if constexpr (MODE != LIN_DW) {
    grp = group_of_row(g.offsets, g.G, g.M, (int)row);
    if (grp >= g.G) {
      if (c % 4 != 0) return;
      linear_zero<ET, MODE>(g, (int)row, c);
      return;
    }
  }
  float z[1][W] = {};
#pragma unroll 4
  for (int s = 0; s < g.splits; ++s) {
    const V v = *(const V*)(g.partial + (s * rows + row) * ldp + c);
#pragma unroll
    for (int j = 0; j < W; ++j) z[0][j] += v[j];
  }
  if constexpr (MODE == LIN_FWD) {
    float b[W] = {};
    const int m[1] = {(int)row};
    const bool ok[1] = {true};
    if (c >= g.N) return;
    if (g.bias) load_w<ET, W, VEC>(static_cast<const ET*>(g.bias) + (long)grp * g.N + c, g.N - c, b);
    with_act(g.act.type, [&](auto act) { linear_rows<ET, decltype(act)::value, W, 1, VEC>(g, z, b, c, m, ok); });
  } else if (c < g.K) store_w<ET, W, VEC>(static_cast<ET*>(g.out) + row * g.K + c, g.K - c, z[0]);
}

// The same for a forward product whose pre-activations leave in 8 bits: a row's
// threads are whole blocks of columns, so that a block's lanes are neighbours.
template <typename ET, bool VEC>
__global__ void __launch_bounds__(256) qmoe_linear_finish8(const LinearGemm g, int b0) {
  constexpr int W = VEC ? 4 : 2;
  typedef float V __attribute__((ext_vector_type(W)));
  const int bl = g.pre8.block_log;
  const long ldp = (g.N + 3) & ~3, per = (((long)g.N + (1 << bl) - 1) >> bl << bl) / W;
  const long i = (long)(b0 + blockIdx.x) * 256 + threadIdx.x, row = i / per;
  const int c = (int)(i - row * per) * W;
  if (row >= g.M) return;
  const int grp = group_of_row(g.offsets, g.G, g.M, (int)row);
  if (grp >= g.G) {
    if (c % 4 != 0) return;
    linear_zero<ET, LIN_FWD>(g, (int)row, c);
    linear_zero8(g.pre8, g.N, (int)row, c);
    return;
  }
  float z[1][W] = {};
  if (c < ldp) {
#pragma unroll 4
    for (int s = 0; s < g.splits; ++s) {
      const V v = *(const V*)(g.partial + ((long)s * g.M + row) * ldp + c);
#pragma unroll
      for (int j = 0; j < W; ++j) z[0][j] += v[j];
    }
  }
  float b[W] = {};
  const int m[1] = {(int)row};
  const bool ok[1] = {true};
  if (g.bias && c < g.N) load_w<ET, W, VEC>(static_cast<const ET*>(g.bias) + (long)grp * g.N + c, g.N - c, b);
  linear_rows8<W, 1>(g, z, b, c, m, ok);
  if (c >= g.N) return;
  with_act(g.act.type, [&](auto act) { linear_rows<ET, decltype(act)::value, W, 1, VEC>(g, z, b, c, m, ok); });
}

template <typename ET>
hipError_t go_finish8(const LinearGemm& g, hipStream_t st) {
  const bool vec = linear_vec<ET>(g, LIN_FWD);
  const long block = 1l << g.pre8.block_log;
  const long n = (long)g.M * ((g.N + block - 1) / block * block / (vec ? 4 : 2));
  return in_launches((n + 255) / 256, [&](int b0, unsigned count) {
    if (vec) hipLaunchKernelGGL((qmoe_linear_finish8<ET, true>), dim3(count), dim3(256), 0, st, g, b0);
    else hipLaunchKernelGGL((qmoe_linear_finish8<ET, false>), dim3(count), dim3(256), 0, st, g, b0);
  });
}

template <typename ET, int MODE>
hipError_t go_finish(const LinearGemm& g, hipStream_t st) {
  const long cols = MODE == LIN_FWD ? g.N : g.K;
  const long rows = MODE == LIN_DW ? (long)g.G * g.N : g.M;
  const bool vec = linear_vec<ET>(g, MODE);
  const long n = rows * ((cols + 3) / 4) * (vec ? 1 : 2);
  const dim3 grid((unsigned)((n + 255) / 256)), block(256);
  if (vec) hipLaunchKernelGGL((qmoe_linear_finish<ET, MODE, true>), grid, block, 0, st, g);
  else hipLaunchKernelGGL((qmoe_linear_finish<ET, MODE, false>), grid, block, 0, st, g);
  return hipGetLastError();
}

template <typename ET>
hipError_t finish_mode(int mode, const LinearGemm& g, hipStream_t st) {
  if (mode == LIN_FWD) return g.pre8.codes ? go_finish8<ET>(g, st) : go_finish<ET, LIN_FWD>(g, st);
  if (mode == LIN_DX) return go_finish<ET, LIN_DX>(g, st);
  return go_finish<ET, LIN_DW>(g, st);
}

// dz of kSumRows rows of one group, W columns a lane (16 bytes where rows
// allow it, VEC), and their column sums: float32, of the unrounded dz, in row
// order (the four wavefronts take every fourth row each and add up in
// wavefront order through LDS).  Four rows of a wavefront are in flight at a
// time.  4096 x 14336 bfloat16, silu: 71 us for 352 MB, 5.0 TB/s; with z in 8 bits
// 59 us for 297 MB; sums alone, 16384 x 4096: 27 us for 126 MB, 4.7 TB/s.
// dz of the 16-bit types is rounded to the type: it is the operand of two
// products on the 16-bit matrix instructions, nine times as fast as the float32
// ones that would take it unrounded.  The products then carry two roundings of
// the same size, their operand's and their own: the root mean square error of
// dx and dW is 0.00235 of the result's in bfloat16 (silu, 4096 x 4096 -> 14336),
// 0.00166 from unrounded dz.
// Z8: the format of z where that is held in 8 bits, else -1.
template <typename ET, int ACT, bool VEC, int Z8>
__global__ void __launch_bounds__(256) qmoe_linear_act_grad(const LinearActGrad g, int ncol, int b0) {
  constexpr int W = VEC ? 16 / (int)sizeof(ET) : 4, R = 4;
  constexpr bool glu = ACT == kActSwiglu;
  constexpr int H = glu ? W / 2 : W;
  __shared__ float red[3][64][W + 1];
  const int b = b0 + (int)blockIdx.x, rb = b / ncol;
  int grp, lo, hi;
  if (!RowBlocks(g.offsets, g.G, g.M, kSumRows).find(rb, grp, lo, hi) || grp >= g.G) return;  // the whole workgroup
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int n = (b % ncol * 64 + lane) * W;
  const int left = g.N - n;  // columns from n on
  const long No = glu ? g.N >> 1 : g.N;
  const int m1 = min(hi, lo + kSumRows);
  const ET* dyp = static_cast<const ET*>(g.dy) + (glu ? n >> 1 : n);
  const ET* zp = static_cast<const ET*>(g.z) + n;
  float sum[W] = {};
  for (int m = lo + wave; m < m1; m += 4 * R) {
    float z[R][W], dy[R][H];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long row = m + 4 * r;
      const bool ok = row < m1 && left > 0;
#pragma unroll
      for (int i = 0; i < H; ++i) dy[r][i] = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) z[r][i] = 0.f;
      if (ok) {
        load_w<ET, H, VEC>(dyp + row * No, glu ? left >> 1 : left, dy[r]);
        if constexpr (ACT != kActIdentity) {
          if constexpr (Z8 >= 0) {
            const int bl = g.z8.block_log;
            const float s = g.z8.scales[row * ((g.N + (1 << bl) - 1) >> bl) + (n >> bl)];
            load_codes<ET, Z8, W>(g.z8.codes + row * g.N + n, left, s, z[r]);
          } else load_w<ET, W, VEC>(zp + row * g.N, left, z[r]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long row = m + 4 * r;
      if (row >= m1) continue;
      float dz[W];
      if constexpr (glu) {
#pragma unroll
        for (int i = 0; i < H; ++i) lin_swiglu_grad<sizeof(ET) == 2>(dy[r][i], z[r][2 * i], z[r][2 * i + 1], g.act, dz[2 * i], dz[2 * i + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) dz[i] = lin_act_grad<sizeof(ET) == 2>(dy[r][i], z[r][i], ACT);
      }
      // (columns from N on have a zero gradient: zeros in dz)
      if (g.dz && n < g.lddz) store_w<ET, W, VEC>(static_cast<ET*>(g.dz) + row * g.lddz + n, (int)g.lddz - n, dz);
#pragma unroll
      for (int i = 0; i < W; ++i) sum[i] += dz[i];
    }
  }
  if (!g.sums) return;
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < W; ++i) red[wave - 1][lane][i] = sum[i];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int w = 0; w < 3; ++w)
#pragma unroll
    for (int i = 0; i < W; ++i) sum[i] += red[w][lane][i];
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (i < left) g.sums[(long)rb * g.N + n + i] = sum[i];
}

template <typename ET>
hipError_t go_act_grad(const LinearActGrad& g, hipStream_t st) {
  auto al = [](const void* p, uintptr_t m) { return (reinterpret_cast<uintptr_t>(p) & m) == 0; };
  const bool glu = g.act.type == kActSwiglu;
  constexpr int W = 16 / (int)sizeof(ET);
  const bool vec = g.N % W == 0 && al(g.z, 15) && al(g.dz, 15) && al(g.dy, glu ? 7 : 15);
  const long blocks = linear_sum_blocks(g.M, g.offsets ? g.G : -1);
  const long cols = g.dz && g.lddz > g.N ? g.lddz : g.N;
  const int per = 64 * (vec ? W : 4);
  const int ncol = (int)((cols + per - 1) / per);
  return in_launches(blocks * ncol, [&](int b0, unsigned count) {
    const dim3 grid(count), block(256);
    with_act(g.act.type, [&](auto act) {
      constexpr int A = decltype(act)::value;
      auto go = [&](auto z8) {
        constexpr int Z = decltype(z8)::value;
        if (vec) hipLaunchKernelGGL((qmoe_linear_act_grad<ET, A, true, Z>), grid, block, 0, st, g, ncol, b0);
        else hipLaunchKernelGGL((qmoe_linear_act_grad<ET, A, false, Z>), grid, block, 0, st, g, ncol, b0);
      };
      if constexpr (A != kActIdentity) {
        if (g.z8.codes) return with_format(g.z8.format, go);
      }
      go(std::integral_constant<int, -1>{});
    });
  });
}

// One column a thread: the group's row blocks in order (14336 columns, 64
// blocks: 5 us).
template <typename ET>
__global__ void __launch_bounds__(256) qmoe_linear_bias_grad(const float* __restrict__ sums,
                                                             const int* __restrict__ offsets, int G, int M, int N,
                                                             int ncol, int nblocks, ET* __restrict__ db) {
  const int grp = blockIdx.x / ncol;
  int first, count;
  group_blocks(offsets, G, M, kSumRows, grp, first, count);
  // (falling offsets: groups overlap, their blocks pass what there is or 31 bits)
  count = first < 0 ? 0 : max(0, min(count, nblocks - first));
  const int n = (blockIdx.x % ncol) * 256 + threadIdx.x;
  if (n >= N) return;
  float s = 0.f;
  const float* p = sums + (long)first * N + n;
#pragma unroll 8
  for (int i = 0; i < count; ++i) s += p[(long)i * N];
  db[(long)grp * N + n] = (ET)s;
}

// cols elements of each row into rows of ld (whole 16-byte pieces), zeros
// behind them: a workgroup a row, a thread a piece (the source pieces are
// aligned to their element only), two operands a launch.  1001 + 1411 rows of
// 2047 float32: 8 us for 40 MB, 5 TB/s.
template <typename U>
__global__ void __launch_bounds__(256) qmoe_linear_pad(LinearPad a, LinearPad b) {
  constexpr int N = 16 / sizeof(U);
  typedef U V __attribute__((ext_vector_type(N)));
  typedef V VU __attribute__((aligned(sizeof(U))));
  for (long i = blockIdx.x; i < a.rows + b.rows; i += gridDim.x) {
    const bool second = i >= a.rows;
    const long r = second ? i - a.rows : i;
    const int cols = (int)(second ? b.cols : a.cols), ld = (int)(second ? b.ld : a.ld);
    const U* src = static_cast<const U*>(second ? b.src : a.src) + r * cols;
    U* dst = static_cast<U*>(second ? b.dst : a.dst) + r * ld;
    for (int c = threadIdx.x * N; c < ld; c += 256 * N) {
      V v;
      if (c + N <= cols) {
        v = *(const VU*)(src + c);
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = c + k < cols ? src[c + k] : (U)0;
      }
      *(V*)(dst + c) = v;
    }
  }
}

}  // namespace

hipError_t launch_linear_finish(int type, int mode, const LinearGemm& g, hipStream_t st) {
  if (type == LIN_F32) return finish_mode<float>(mode, g, st);
  if (type == LIN_F16) return finish_mode<_Float16>(mode, g, st);
  return finish_mode<__bf16>(mode, g, st);
}

hipError_t launch_linear_act_grad(int type, const LinearActGrad& g, hipStream_t st) {
  if (type == LIN_F32) return go_act_grad<float>(g, st);
  if (type == LIN_F16) return go_act_grad<_Float16>(g, st);
  return go_act_grad<__bf16>(g, st);
}

hipError_t launch_linear_bias_grad(int type, const float* sums, const int* offsets, int G, int M, int N, void* db,
                                   hipStream_t st) {
  const int ncol = (N + 255) / 256, nblocks = (int)linear_sum_blocks(M, offsets ? G : -1);
  const dim3 grid((unsigned)((long)G * ncol)), block(256);
  if (type == LIN_F32)
    hipLaunchKernelGGL(qmoe_linear_bias_grad<float>, grid, block, 0, st, sums, offsets, G, M, N, ncol, nblocks, (float*)db);
  else if (type == LIN_F16)
    hipLaunchKernelGGL(qmoe_linear_bias_grad<_Float16>, grid, block, 0, st, sums, offsets, G, M, N, ncol, nblocks, (_Float16*)db);
  else
    hipLaunchKernelGGL(qmoe_linear_bias_grad<__bf16>, grid, block, 0, st, sums, offsets, G, M, N, ncol, nblocks, (__bf16*)db);
  return hipGetLastError();
}

hipError_t launch_linear_pad(int esize, const LinearPad& a, const LinearPad& b, hipStream_t st) {
  const long rows = a.rows + b.rows;
  if (rows == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<long>(rows, 1 << 20)), block(256);
  if (esize == 4) hipLaunchKernelGGL(qmoe_linear_pad<uint32_t>, grid, block, 0, st, a, b);
  else hipLaunchKernelGGL(qmoe_linear_pad<uint16_t>, grid, block, 0, st, a, b);
  return hipGetLastError();
}

hipError_t launch_linear_f16(int mode, int tile, const LinearGemm& g, hipStream_t st);
hipError_t launch_linear_bf16(int mode, int tile, const LinearGemm& g, hipStream_t st);
hipError_t launch_linear_f32(int mode, int tile, const LinearGemm& g, hipStream_t st);

hipError_t launch_linear(int type, int mode, int tile, const LinearGemm& g, hipStream_t st) {
  if (type == LIN_F32) return launch_linear_f32(mode, tile, g, st);
  if (type == LIN_F16) return launch_linear_f16(mode, tile, g, st);
  return launch_linear_bf16(mode, tile, g, st);
}

}  // namespace qmoe
