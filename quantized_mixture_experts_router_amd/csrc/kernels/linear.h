// Linear layers (dense, or one weight per group of consecutive rows) and
// their gradients: launch functions (host side; enqueue only).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmoe {

enum LinearType { LIN_F32 = 0, LIN_F16 = 1, LIN_BF16 = 2 };

// Which product: the operands are rows of q (output rows) and rows or
// columns of p (output columns), summed over r.
//   LIN_FWD  z  [M, N] = x  [M, K] . w [N, K]^T     q = x rows,   p = w rows,    r = K
//   LIN_DX   dx [M, K] = dz [M, N] . w [N, K]       q = dz rows,  p = w columns, r = N
//   LIN_DW   dw [N, K] = dz [M, N]^T . x [M, K]     q = dz cols,  p = x columns, r = the group's rows
enum LinearMode { LIN_FWD = 0, LIN_DX = 1, LIN_DW = 2 };

struct LinearAct {
  int type;  // qmoe_activation
  float alpha, beta;
  int has_limit;
  float limit;
};

struct LinearGemm {
  const void* x;   // [M][ldx]
  const void* w;   // [G][N][ldw]
  const void* dz;  // [M][lddz] (LIN_DX, LIN_DW)
  long ldx, ldw, lddz;  // row strides in elements, whole 16-byte runs; 16-byte aligned pointers
  const int* offsets;   // [G + 1] first row of each group; NULL: one group of all rows
  int G, M, N, K;
  const void* bias;  // [G][N] or NULL   (LIN_FWD)
  const void* res;   // [M][ldo] or NULL (LIN_FWD)
  void* pre;         // [M][N] or NULL   (LIN_FWD)
  void* out;         // [M][No], dx [M][K] or dw [G][N][K]
  float* partial;    // splits > 1: [splits][rows of out][cols4] fp32 sums
  int splits;        // ranges of r
  LinearAct act;
};

// Tile shapes of the matrix kernel (rows of q by rows / columns of p).
enum LinearTile { LT_256x256 = 0, LT_128x128 = 1, LT_64x128 = 2, LT_32x128 = 3 };
struct LinearPlan {
  int tile;    // LinearTile
  int splits;  // ranges of r (1: the matrix kernel finishes the output)
};
hipError_t launch_linear(int type, int mode, int tile, const LinearGemm& g, hipStream_t st);
// Sum of the ranges of r and the epilogue (splits > 1).
hipError_t launch_linear_finish(int type, int mode, const LinearGemm& g, hipStream_t st);

// dz = dy * act'(z) (rows of the groups only) into dz [M][lddz], columns from
// N on zeroed, and the column sums of each row block into sums (kSumRows rows
// of a group each, [blocks][N]); dz or sums may be NULL.  z is NULL for the
// identity.
constexpr int kSumRows = 64;
// Row blocks of M rows in G groups (G < 0: no groups), at most.
constexpr long linear_sum_blocks(long M, long G) { return (M + kSumRows - 1) / kSumRows + (G < 0 ? 0 : G + 1); }
struct LinearActGrad {
  const void* dy;  // [M][No]
  const void* z;   // [M][N]
  void* dz;
  long lddz;
  float* sums;
  const int* offsets;
  int G, M, N;
  LinearAct act;
};
hipError_t launch_linear_act_grad(int type, const LinearActGrad& g, hipStream_t st);
// db[g][n] = sum of the row blocks' column sums of group g, in row order.
hipError_t launch_linear_bias_grad(int type, const float* sums, const int* offsets, int G, int M, int N, void* db,
                                   hipStream_t st);
// rows x cols elements -> rows of ld elements (whole 16-byte runs, 16-byte
// aligned), zeros from cols on; two operands (rows 0: none).
struct LinearPad {
  const void* src;
  long rows, cols;
  void* dst;
  long ld;
};
hipError_t launch_linear_pad(int esize, const LinearPad& a, const LinearPad& b, hipStream_t st);

}  // namespace qmoe
