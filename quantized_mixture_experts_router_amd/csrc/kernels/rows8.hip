// Rows to 8 bits and back (rows8.h).  Both are bound by HBM.
#include "launches.h"
#include "rows8.hpp"
#include "tokens.h"

namespace qmoe {

namespace {

constexpr int kR = 4;  // rows of a thread, in flight together

// A thread per piece of W columns (16 bytes) of kR rows, `per` threads a row (a
// power of two up to 256, the rest of the row in blockIdx.y): the lanes of one
// block of columns, neighbours in a wavefront, find its largest magnitude.
template <typename ET, int F>
__global__ void __launch_bounds__(256) qmoe_quantize_rows(const ET* __restrict__ x, long M, int N, int block_log,
                                                          int per_log, int b0, uint8_t* __restrict__ codes,
                                                          float* __restrict__ scales) {
  constexpr int W = 16 / (int)sizeof(ET), WL = W == 8 ? 3 : 2;
  const int c = (((int)blockIdx.y << per_log) + ((int)threadIdx.x & ((1 << per_log) - 1))) * W;
  const long step = 1l << (8 - per_log);
  const long m0 = (long)(b0 + blockIdx.x) * (step * kR) + (threadIdx.x >> per_log);
  const int n = N - c;
  const int blocks = (N + (1 << block_log) - 1) >> block_log;
  typename RowPiece<ET, W>::type t[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const long m = m0 + r * step;
    t[r] = typename RowPiece<ET, W>::type{};
    if (m < M && n > 0) t[r] = load_piece<ET, W>(x + m * N + c, n);
  }
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const long m = m0 + r * step;
    float v[W];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      v[i] = (float)t[r][i];
      top = max(top, abs_bits(v[i]));
    }
    top = lanes_max(top, block_log - WL);
    const uint32_t s = r8_scale_bits<F>(top);
    if (m >= M || n <= 0) continue;
    store_codes<F, W>(codes + m * N + c, n, v, r8_inverse(s));
    if ((c & ((1 << block_log) - 1)) == 0) scales[m * blocks + (c >> block_log)] = __uint_as_float(s);
  }
}

// A thread per piece of W columns of kR output rows, as above.
template <typename ET, int F>
__global__ void __launch_bounds__(256) qmoe_dequantize_rows(const uint8_t* __restrict__ codes,
                                                            const float* __restrict__ scales,
                                                            const int* __restrict__ perm, int k, long M, int N,
                                                            int block_log, int per_log, int b0, ET* __restrict__ out,
                                                            long ld) {
  constexpr int W = 16 / (int)sizeof(ET);
  const int c = (((int)blockIdx.y << per_log) + ((int)threadIdx.x & ((1 << per_log) - 1))) * W;
  const long step = 1l << (8 - per_log);
  const long m0 = (long)(b0 + blockIdx.x) * (step * kR) + (threadIdx.x >> per_log);
  if (c >= ld) return;
  const int n = N - c;
  const int blocks = (N + (1 << block_log) - 1) >> block_log;
  long src[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const long m = m0 + r * step;
    src[r] = m;
    if (perm) {
      const int p = m < M ? perm[m] : -1;
      src[r] = p >= 0 && p < M ? (long)((uint32_t)p / (uint32_t)k) : -1;
    } else if (m >= M) src[r] = -1;
  }
  typename RowPiece<uint8_t, W>::type t[kR];
  float s[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    t[r] = typename RowPiece<uint8_t, W>::type{};
    s[r] = 0.f;
    if (src[r] >= 0 && n > 0) {
      t[r] = load_piece<uint8_t, W>(codes + src[r] * N + c, n);
      s[r] = scales[src[r] * blocks + (c >> block_log)];
    }
  }
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const long m = m0 + r * step;
    if (m >= M) continue;
    uint32_t u[W / 4];
    __builtin_memcpy(u, &t[r], W);
    float v[W];
#pragma unroll
    for (int i = 0; i < W / 4; ++i) r8_decode4<F>(u[i], s[r], v + 4 * i);
    if (r8_may_pass<ET, F>(s[r])) {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = r8_limit<ET>(v[i]);
    }
    typename RowPiece<ET, W>::type o;
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = (ET)(i < n && src[r] >= 0 ? v[i] : 0.f);
    store_piece<ET, W>(out + m * ld + c, (int)min(ld - c, (long)W), o);
  }
}

// Threads a row (log2), launches' workgroups and the rest of the row in y.
struct PieceGrid {
  int per_log;
  long x;
  unsigned y;
};
PieceGrid piece_grid(long M, long pieces, int least) {
  int l = least;
  while (l < 8 && (1l << l) < pieces) ++l;
  const long rows = kR << (8 - l);
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
hipError_t dequantize_t(const Rows8& q, const int* perm, int k, long M, long N, void* out, long ld, hipStream_t st) {
  constexpr int W = 16 / (int)sizeof(ET);
  const PieceGrid g = piece_grid(M, (ld + W - 1) / W, 0);
  return in_launches(g.x, [&](int b0, unsigned n) {
    with_format(q.format, [&](auto f) {
      hipLaunchKernelGGL((qmoe_dequantize_rows<ET, decltype(f)::value>), dim3(n, g.y), dim3(256), 0, st, q.codes, q.scales, perm, k, M, (int)N, q.block_log, g.per_log, b0, (ET*)out, ld);
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
                                  hipStream_t st) {
  if (type == ROW_F32) return dequantize_t<float>(q, perm, k, M, N, out, ld, st);
  if (type == ROW_F16) return dequantize_t<_Float16>(q, perm, k, M, N, out, ld, st);
  return dequantize_t<__bf16>(q, perm, k, M, N, out, ld, st);
}

}  // namespace qmoe
