// Rows to 8 bits and back (rows8.h).  Both are bound by HBM.
#include "launches.h"
#include "rows8.hpp"
#include "tokens.h"

namespace qmoe {

namespace {

// A thread per piece of W columns (16 bytes), `per` threads a row (a power of two
// up to 256, the rest of the row in blockIdx.y): the lanes of one block of columns,
// neighbours in a wavefront, find its largest magnitude.
// 4096 x 14336 bfloat16: 30 to 33 us for 178 MB, 5.4 to 5.9 TB/s; 16 x 4096: 2.5 us.
// One row a thread: two, four and eight rows in flight took 5, 7 and 9 % longer there
// and 2.5, 3.2 and 4.6 us against 2.2 here.
template <typename ET, int F>
__global__ void __launch_bounds__(256) qmoe_quantize_rows(const ET* __restrict__ x, long M, int N, int block_log,
                                                          int per_log, int b0, uint8_t* __restrict__ codes,
                                                          float* __restrict__ scales) {
  constexpr int W = 16 / (int)sizeof(ET), WL = W == 8 ? 3 : 2;
  const int c = (((int)blockIdx.y << per_log) + ((int)threadIdx.x & ((1 << per_log) - 1))) * W;
  const long m = ((long)(b0 + blockIdx.x) << (8 - per_log)) + (threadIdx.x >> per_log);
  const int n = N - c;
  const bool here = m < M && n > 0;
  typename RowPiece<ET, W>::type t = {};
  if (here) t = load_piece<ET, W>(x + m * N + c, n);
  float v[W];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    v[i] = (float)t[i];
    top = max(top, abs_bits(v[i]));
  }
  const uint32_t s = r8_scale_bits<F>(lanes_max(top, block_log - WL));
  if (!here) return;
  store_codes<F, W>(codes + m * N + c, n, v, r8_inverse(s));
  const int blocks = (N + (1 << block_log) - 1) >> block_log;
  if ((c & ((1 << block_log) - 1)) == 0) scales[m * blocks + (c >> block_log)] = __uint_as_float(s);
}

// A thread per piece of W columns of an output row, as above.  4096 x 14336 to
// bfloat16: 27 us for 178 MB, 36 (5.0 TB/s) with nothing of them in the caches; 2047
// rows of 2048 to 12282 float16 rows 13.7 us, where 50 MB are written, at 3.7 TB/s, and 4 read.
template <typename ET, int F>
__global__ void __launch_bounds__(256) qmoe_dequantize_rows(const uint8_t* __restrict__ codes,
                                                            const float* __restrict__ scales,
                                                            const int* __restrict__ perm, int k, long M, int N,
                                                            int block_log, int per_log, int b0, int stream,
                                                            ET* __restrict__ out, long ld) {
  constexpr int W = 16 / (int)sizeof(ET);
  const int c = (((int)blockIdx.y << per_log) + ((int)threadIdx.x & ((1 << per_log) - 1))) * W;
  const long m = ((long)(b0 + blockIdx.x) << (8 - per_log)) + (threadIdx.x >> per_log);
  if (m >= M || c >= ld) return;
  const int n = N - c;
  long src = m;
  if (perm) {
    const int p = perm[m];
    src = p >= 0 && p < M ? (long)((uint32_t)p / (uint32_t)k) : -1;
  }
  float v[W] = {};
  if (src >= 0 && n > 0) {
    const int blocks = (N + (1 << block_log) - 1) >> block_log;
    load_codes<ET, F, W>(codes + src * N + c, n, scales[src * blocks + (c >> block_log)], v);
  }
  typename RowPiece<ET, W>::type o;
#pragma unroll
  for (int i = 0; i < W; ++i) o[i] = (ET)v[i];
  store_piece<ET, W>(out + m * ld + c, (int)min(ld - c, (long)W), o, stream);
}

// Threads a row (log2, at least `least`), launches' workgroups and the rest of
// the row in y.
struct PieceGrid {
  int per_log;
  long x;
  unsigned y;
};
PieceGrid piece_grid(long M, long pieces, int least) {
  int l = least;
  while (l < 8 && (1l << l) < pieces) ++l;
  const long rows = 1l << (8 - l);
  return {l, (M + rows - 1) / rows, (unsigned)((pieces + (1l << l) - 1) >> l)};
}

template <typename ET>
hipError_t quantize_t(const void* x, long M, long N, const Rows8& q, hipStream_t st) {
  constexpr int W = 16 / (int)sizeof(ET), WL = W == 8 ? 3 : 2;
  // (a row's threads are whole blocks of columns)
  const PieceGrid g = piece_grid(M, (N + W - 1) / W, q.block_log - WL);
  return in_launches(g.x, [&](int b0, unsigned n) {
    with_format(q.format, [&](auto f) {
      hipLaunchKernelGGL((qmoe_quantize_rows<ET, decltype(f)::value>), dim3(n, g.y), dim3(256), 0, st, (const ET*)x, M, (int)N, q.block_log, g.per_log, b0, q.codes, q.scales);
    });
  });
}

template <typename ET>
hipError_t dequantize_t(const Rows8& q, const int* perm, int k, long M, long N, void* out, long ld, bool soon,
                        hipStream_t st) {
  constexpr int W = 16 / (int)sizeof(ET);
  const PieceGrid g = piece_grid(M, (ld + W - 1) / W, 0);
  return in_launches(g.x, [&](int b0, unsigned n) {
    with_format(q.format, [&](auto f) {
      hipLaunchKernelGGL((qmoe_dequantize_rows<ET, decltype(f)::value>), dim3(n, g.y), dim3(256), 0, st, q.codes, q.scales, perm, k, M, (int)N, q.block_log, g.per_log, b0, !soon && M * ld * (long)sizeof(ET) >= kStreamBytes, (ET*)out, ld);
    });
  });
}

}  // namespace

hipError_t launch_quantize_rows(int type, const void* x, long M, long N, const Rows8& q, hipStream_t st) {
  if (type == ROW_F32) return quantize_t<float>(x, M, N, q, st);
  if (type == ROW_F16) return quantize_t<_Float16>(x, M, N, q, st);
  return quantize_t<__bf16>(x, M, N, q, st);
}

hipError_t launch_dequantize_rows(int type, const Rows8& q, const int* perm, int k, long M, long N, void* out, long ld,
                                  bool soon, hipStream_t st) {
  if (type == ROW_F32) return dequantize_t<float>(q, perm, k, M, N, out, ld, soon, st);
  if (type == ROW_F16) return dequantize_t<_Float16>(q, perm, k, M, N, out, ld, soon, st);
  return dequantize_t<__bf16>(q, perm, k, M, N, out, ld, soon, st);
}

}  // namespace qmoe
