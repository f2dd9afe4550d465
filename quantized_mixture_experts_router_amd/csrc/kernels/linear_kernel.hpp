// The matrix kernel of the linear layers (LinearGemm in linear.h).
//
//   out[q][p] = sum_r Q(q, r) P(p, r)
//
// Each operand is either a run of r per row (x and w of the forward product,
// dz of dx) or a run of q or p per r (w of dx; dz and x of dw).  Both arrive
// in LDS as they lie in memory, 16 bytes a lane straight from HBM
// (buffer loads to LDS: the buffer's size is the operand's own, so a row past
// the group's end or a column past the row's reads as zero without a branch),
// and a stage holds 128 bytes of r per row of a run-of-r operand (64 16-bit or
// 32 32-bit values) or as many r rows of the other kind.  Pieces of 16 bytes
// are permuted inside their row (the source address is; the LDS side of the
// load is linear) so that the lanes that read together meet different banks:
//  - run-of-r tiles, 128-byte rows, sixteen lanes read one piece of sixteen
//    rows: piece c of row i in slot c ^ (i / 2 & 7);
//  - the other kind, 16-bit: the transposing LDS read gives a lane four r of
//    its column; its half-wavefronts read 32 bytes of rows r .. r + 3 and
//    r + 8 .. r + 11: slot c ^ (4 (r & 3) + 2 (r / 8 & 1));
//  - 32-bit values of the other kind are read one by one, 64 bytes of rows
//    r, r + 4, r + 8, r + 12: slot c ^ 4 (r / 4 & 3).
//
// The matrix instructions are the 16-row ones: at the card's power limit they
// sustain 2.1 GHz where the 32-row ones do 1.8 (2170 against 1900 TFLOP/s in
// registers).  Their row operand is P and their column operand Q, so a lane
// ends with four consecutive output columns of one output row.
#pragma once
#include <type_traits>

#include "launches.h"
#include "linear_common.hpp"

namespace qmoe {

template <typename ET>
struct LinMma {  // 16-bit: 16 x 16 x 32, eight r a lane
  using Frag = typename std::conditional<std::is_same<ET, _Float16>::value, h16x8, b16x8>::type;
  static __device__ __forceinline__ f32x4 mma(Frag p, Frag q, f32x4 c) {
    if constexpr (std::is_same<ET, _Float16>::value) return __builtin_amdgcn_mfma_f32_16x16x32_f16(p, q, c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, q, c, 0, 0, 0);
  }
};
template <>
struct LinMma<float> {  // 16 x 16 x 4, four steps over the four r a lane holds
  using Frag = f32x4;
  static __device__ __forceinline__ f32x4 mma(Frag p, Frag q, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(p[j], q[j], c, 0, 0, 0);
    return c;
  }
};

// Wait until at most N vector-memory operations of this wavefront are in
// flight and its LDS accesses are done.
template <int N>
__device__ __forceinline__ void lin_wait() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4));
  asm volatile("" ::: "memory");
}

// helper lambdas are always inlined (what they capture stays in registers)
#define QMOE_INLINE __attribute__((always_inline))
#define QMOE_LDS(p) ((__attribute__((address_space(3))) void*)(p))

// 16 bytes a lane from buffer rs at vo + so into LDS at dst + 16 lane (the
// instruction has no register output).  Written out because the compiler
// takes every transposing LDS read for a reader of the loads in flight and
// would wait for all of them in front of each; the waits are lin_wait's.
__device__ __forceinline__ void load_lds16(u32x4 rs, uint32_t dst, int vo, int so) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(dst),
      "v"(vo), "s"(rs), "s"(so)
      : "memory", "m0");
}

// One operand's tile of BT rows or columns: fills a stage and reads fragments.
//   RUN: rows of consecutive r.  else: r rows of consecutive columns.
template <typename ET, int BT, bool RUN, int NW>
struct LinOperand {
  static constexpr int ES = sizeof(ET), EPC = 16 / ES, BK = 128 / ES;
  static constexpr int kBytes = BT * 128;            // one stage
  static constexpr int kLoads = kBytes / 1024 / NW;  // load instructions of a wavefront and stage
  static constexpr int CPR = BT * ES / 16;           // pieces per r row
  static constexpr int RPI = RUN ? 8 : 64 / CPR;     // rows one instruction covers
  // the permutation depends on r mod 16: lane offsets that repeat over a
  // wavefront's instructions
  static constexpr int kOffs = RUN || RPI * NW >= 16 ? 1 : 16 / (RPI * NW);
  static_assert(kBytes % (1024 * NW) == 0 && NW % 2 == 0, "every wavefront issues the same count");
  static_assert(kLoads % kOffs == 0 || kLoads < kOffs, "the offsets repeat");
  static constexpr int kOut = (int)0x80000000;  // an offset past every buffer

  const char* base;  // stage's first row or column, at the stage's first r
  long left;         // bytes from base to the end of the operand's rows
  int ldb;           // row stride in bytes
  int voff[kOffs];   // this lane's offset in an instruction's rows
  int piece;         // RUN: first r of this lane's piece in its stage

  static __device__ __forceinline__ int swz(int r) {
    if constexpr (ES == 4) return CPR >= 16 ? ((r >> 2) & 3) << 2 : ((r >> 2) & 1) << 2;
    const int h = ((r >> 3) & 1) << 1;
    if constexpr (CPR >= 16) return ((r & 3) << 2) | h;
    if constexpr (CPR == 8) return (((r >> 1) & 1) << 2) | h;  // 128-byte rows: neighbours already differ
    return h;                                                  // 64-byte rows: four differ by themselves
  }

  // src: element (0, 0) of the tile; ld: row stride in elements; rows: RUN,
  // valid rows, else valid r; row_len: elements from src to its row's end;
  // cols: else, valid columns from the tile's first; kb: first stage
  __device__ __forceinline__ void init(const ET* src, long ld, long rows, long row_len, int cols, long kb, int wave,
                                       int lane) {
    ldb = (int)(ld * ES);
    const long at = kb * (RUN ? 128 : (long)BK * ldb);
    if (RUN && rows > BT) rows = BT;  // (the tile's rows stay within 32 bits)
    base = reinterpret_cast<const char*>(src) + at;
    left = rows > 0 ? ((rows - 1) * ld + row_len) * ES - at : 0;
    if constexpr (RUN) {
      // row / 2 of row 8 (i NW + wave) + lane / 8, NW even
      const int c = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));
      piece = c * EPC;
      voff[0] = (lane >> 3) * ldb + c * 16;
    } else {
      piece = 0;
#pragma unroll
      for (int i = 0; i < kOffs; ++i) {
        const int c = (lane % CPR) ^ swz((i * NW + wave) * RPI + lane / CPR);
        voff[i] = c * EPC < cols ? lane / CPR * ldb + c * 16 : kOut;
      }
    }
  }

  // Load instruction i of the next stage into LDS at dst; r0 = the stage's
  // first r (of R); not on: past the range of r, nothing is read and the
  // stage fills with zeros.
  __device__ __forceinline__ void load(int i, char* dst, int r0, int R, bool on, int wave) const {
    const long rem = on ? left : 0;
    const int size = RUN ? max((int)rem, 0) : (int)(rem < 0 ? 0 : rem > 0x7fffffff ? 0x7fffffff : rem);
    const uint64_t at = (uint64_t)base;
    const u32x4 rs = {(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, (uint32_t)size, 0x00027000u};
    const int idx = i * NW + wave;
    // the last stage: pieces from R on are out of range, not the next row
    int vo = RUN && r0 + piece >= R ? kOut : voff[0];
    if constexpr (kOffs > 1) vo = voff[i % kOffs];
    load_lds16(rs, (uint32_t)(uintptr_t)QMOE_LDS(dst + idx * 1024), vo, idx * RPI * ldb);
  }
  __device__ __forceinline__ void next() {
    const long step = RUN ? 128 : (long)BK * ldb;
    base += step;
    left -= step;
  }
  __device__ __forceinline__ void rewind(int stages) {
    const long back = stages * (RUN ? 128 : (long)BK * ldb);
    base -= back;
    left += back;
  }

  // This lane's operand of k step ks (32 16-bit or 16 32-bit r) for the 16
  // rows or columns from t0 on: r = 8 (lane / 16) .. + 7 of the step (32-bit:
  // 4 (lane / 16) .. + 3).
  static __device__ __forceinline__ typename LinMma<ET>::Frag frag(const char* src, int t0, int ks, int lane) {
    using Frag = typename LinMma<ET>::Frag;
    if constexpr (RUN) {
      const int c = 4 * ks + (lane >> 4);
      return *(const Frag*)(src + (t0 + (lane & 15)) * 128 + ((c ^ ((lane >> 1) & 7)) << 4));
    } else if constexpr (ES == 4) {
      Frag f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 16 * ks + 4 * (lane >> 4) + j;
        const int c = ((t0 >> 2) + ((lane & 15) >> 2)) ^ swz(r);
        f[j] = *(const float*)(src + r * (BT * 4) + (c << 4) + (lane & 3) * 4);
      }
      return f;
    } else {
      union {
        s16x4 h[2];
        Frag f;
      } u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 32 * ks + 8 * (lane >> 4) + 4 * h + ((lane & 15) >> 2);
        const int c = ((t0 >> 3) + ((lane & 3) >> 1)) ^ swz(r);
        u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(src + r * (BT * 2) + (c << 4) + (lane & 1) * 8));
      }
      return u.f;
    }
  }
};

template <typename ET, int MODE, int BQ, int BP, int WQ, int WP, int NST, bool VEC, bool TURN>
__global__ void __launch_bounds__(64 * WQ * WP) qmoe_linear(const LinearGemm g, int nq, int np, int b0) {
  constexpr int NW = WQ * WP, TQ = BQ / WQ / 16, TP = BP / WP / 16;
  using OP = LinOperand<ET, BP, MODE == LIN_FWD, NW>;
  using OQ = LinOperand<ET, BQ, MODE != LIN_DW, NW>;
  constexpr int BK = OP::BK, KS = 2;
  __shared__ __attribute__((aligned(1024))) char lds[NST][OP::kBytes + OQ::kBytes];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const int ks_id = blockIdx.y;  // range of r
  // (in rows of groups only the device knows how many blocks there are; falling
  // offsets make groups overlap, and the host's bound keeps the walk over
  // the tiles within 32 bits)
  const RowBlocks blocks(MODE == LIN_DW ? nullptr : g.offsets, g.G, g.M, BQ);
  if (MODE != LIN_DW && g.offsets) nq = min(blocks.total, nq);
  if (nq <= 0) return;
  const LinearTileAt tile = linear_tile_of(b0 + blockIdx.x, nq, np);
  const int qb = tile.q, pb = tile.p;
  const int p0 = pb * BP;
  int grp, lo, hi, q0, qrows;  // group, its rows from the tile on, first output row, valid rows of the tile
  const int pcols = MODE == LIN_FWD ? g.N : g.K;
  if (p0 >= pcols) return;
  OP op;
  OQ oq;
  int R;
  if constexpr (MODE == LIN_DW) {
    const int nqg = (g.N + BQ - 1) / BQ;  // q blocks of a group
    grp = qb / nqg;
    if (grp >= g.G) return;
    q0 = (qb - grp * nqg) * BQ;
    qrows = g.N - q0;
    group_rows(g.offsets, g.G, g.M, grp, lo, hi);
    R = hi - lo;
  } else {
    if (!blocks.find(qb, grp, lo, hi)) return;
    q0 = lo;
    qrows = hi - lo;
    if (grp == g.G && g.offsets) {  // rows behind the last group: zeros
      if (ks_id > 0 || g.splits > 1) return;  // (the finishing pass writes them)
      for (int i = threadIdx.x; i < min(qrows, BQ) * (BP / 4); i += 64 * NW) {
        const int m = q0 + i / (BP / 4), c = p0 + 4 * (i % (BP / 4));
        linear_zero<ET, MODE>(g, m, c);
      }
      return;
    }
    R = MODE == LIN_FWD ? g.K : g.N;
  }
  // stages [kb, kb + nk) of this range
  const int nk_all = (R + BK - 1) / BK;
  const int kb = (int)((long)nk_all * ks_id / g.splits);
  const int nk = (int)((long)nk_all * (ks_id + 1) / g.splits) - kb;
  // TURN: the range is walked as a ring, every group's tiles from a stage of
  // their own on (in a product of one q block every tile).  Rows that lie a
  // power of two apart put a stage's pieces into few of the memory's channels,
  // and tiles in step all ask for the same ones: one row by 28672 x 4096 takes
  // 41 us turned and 51 us in step, 128 rows 65 and 71 us, 12288 rows in 64
  // groups by 2816 x 2048 279 and 292 us.  A group's tiles stay in step, since
  // they share its rows (8 groups of 64 rows by 14336 x 4096: 182 us, 188 us with
  // every tile on its own); so do all tiles of other dense products, which
  // would lose 1 % to the bookkeeping.
  int ka = TURN && nk > 0 ? kb + 5 * (g.offsets ? grp : pb) % nk : kb;  // the stage to load next
  if constexpr (MODE == LIN_DW) {
    op.init(static_cast<const ET*>(g.x) + (long)lo * g.ldx + p0, g.ldx, R, g.ldx - p0, g.K - p0, ka, wave, lane);
    oq.init(static_cast<const ET*>(g.dz) + (long)lo * g.lddz + q0, g.lddz, R, g.lddz - q0, g.N - q0, ka, wave, lane);
  } else if constexpr (MODE == LIN_FWD) {
    op.init(static_cast<const ET*>(g.w) + ((long)grp * g.N + p0) * g.ldw, g.ldw, g.N - p0, g.ldw, 0, ka, wave, lane);
    oq.init(static_cast<const ET*>(g.x) + (long)lo * g.ldx, g.ldx, qrows, g.ldx, 0, ka, wave, lane);
  } else {
    op.init(static_cast<const ET*>(g.w) + (long)grp * g.N * g.ldw + p0, g.ldw, g.N, g.ldw - p0, g.K - p0, ka, wave, lane);
    oq.init(static_cast<const ET*>(g.dz) + (long)lo * g.lddz, g.lddz, qrows, g.lddz, 0, ka, wave, lane);
  }

  f32x4 acc[TP][TQ];
#pragma unroll
  for (int a = 0; a < TP; ++a)
#pragma unroll
    for (int b = 0; b < TQ; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int wq = wave / WP, wp = wave % WP;
  // float32: the sums of every kFold stages (256 r) are added up on their own,
  // which keeps a long sum's error at that of its pieces (root mean square of
  // the error over the result's, normal operands, 1024 / 8192 / 32768 terms:
  // 2.9e-7 / 3.0e-7 / 3.2e-7, in one sum 5.7e-7 / 1.1e-6 / 2.3e-6)
  constexpr int kFold = sizeof(ET) == 4 ? 8 : 0;
  f32x4 sum[kFold ? TP : 1][kFold ? TQ : 1];
  if constexpr (kFold > 0) {
#pragma unroll
    for (int a = 0; a < TP; ++a)
#pragma unroll
      for (int b = 0; b < TQ; ++b) sum[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  auto fold = [&]() QMOE_INLINE {
    if constexpr (kFold > 0) {
#pragma unroll
      for (int a = 0; a < TP; ++a)
#pragma unroll
        for (int b = 0; b < TQ; ++b) {
          sum[a][b] += acc[a][b];
          acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }
  };

  // Load instruction i of stage kt into place u (= kt % NST); past the range's
  // end zeros, so that the count of loads in flight stays the same.
  constexpr int kStage = OP::kLoads + OQ::kLoads;
  auto load = [&](int i, int kt, int u) QMOE_INLINE {
    const int at = TURN ? ka : kb + kt;
    if (i < OP::kLoads) op.load(i, lds[u], at * BK, R, kt < nk, wave);
    else oq.load(i - OP::kLoads, lds[u] + OP::kBytes, at * BK, R, kt < nk, wave);
    if (i == kStage - 1) {
      op.next();
      oq.next();
      if (TURN && ++ka == kb + nk) {
        ka = kb;
        op.rewind(nk);
        oq.rewind(nk);
      }
    }
  };
  using Frag = typename LinMma<ET>::Frag;
  Frag fp[2][TP], fq[TQ];
  auto read_p = [&](int a, int u, int ks) QMOE_INLINE { fp[ks][a] = OP::frag(lds[u], (wp * TP + a) * 16, ks, lane); };
  auto read_q = [&](int b, int u, int ks) QMOE_INLINE {
    fq[b] = OQ::frag(lds[u] + OP::kBytes, (wq * TQ + b) * 16, ks, lane);
  };
  // This wavefront's loads of all but the newest NST - 2 stages have landed,
  // its LDS reads are done; then everyone's.
  auto barrier = [&]() QMOE_INLINE {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  };
  auto meet = [&]() QMOE_INLINE {
    lin_wait<(NST - 2) * kStage>();
    barrier();
  };
  // A stage is two k steps; a step runs its matrix instructions block by
  // block (the TP products of one q fragment).  The next step's operands are
  // read meanwhile: a q fragment into its own registers when its block is
  // done, the p fragments into a second set.  In the stage's second step all
  // of the stage has been read, so behind the first block (which covers the
  // last reads; one block later cost 3 %) the workgroup meets; behind the barrier the reads go to the
  // next stage and this stage's place is filled anew, NST stages ahead, a few
  // loads a block.  The scheduling barriers keep that order.
  constexpr int kFill = (kStage + TQ - 1) / TQ;  // loads a block
  constexpr int kPer = (TP + TQ - 1) / TQ;       // p reads a block
  auto block = [&](int b, int ks) QMOE_INLINE {
#pragma unroll
    for (int a = 0; a < TP; ++a) acc[a][b] = LinMma<ET>::mma(fp[ks][a], fq[b], acc[a][b]);
  };
#pragma unroll
  for (int s = 0; s < NST - 1; ++s)
#pragma unroll
    for (int i = 0; i < kStage; ++i) load(i, s, s);
  if (nk > 0) {
    meet();
#pragma unroll
    for (int i = 0; i < kStage; ++i) load(i, NST - 1, NST - 1);
#pragma unroll
    for (int a = 0; a < TP; ++a) read_p(a, 0, 0);
#pragma unroll
    for (int b = 0; b < TQ; ++b) read_q(b, 0, 0);
    for (int kt = 0; kt < nk; kt += NST) {
#pragma unroll
      for (int u = 0; u < NST; ++u) {
        if (kt + u >= nk) break;
#pragma unroll
        for (int b = 0; b < TQ; ++b) {
          block(b, 0);
          __builtin_amdgcn_sched_barrier(0);
          read_q(b, u, 1);
#pragma unroll
          for (int a = b * kPer; a < (b + 1) * kPer && a < TP; ++a) read_p(a, u, 1);
        }
#pragma unroll
        for (int b = 0; b < TQ; ++b) {
          block(b, 1);
          __builtin_amdgcn_sched_barrier(0);
          if (b == 0) meet();
          const int n = (u + 1) % NST;
          read_q(b, n, 0);
#pragma unroll
          for (int a = b * kPer; a < (b + 1) * kPer && a < TP; ++a) read_p(a, n, 0);
#pragma unroll
          for (int i = b * kFill; i < (b + 1) * kFill && i < kStage; ++i) load(i, kt + u + NST, u);
        }
        if constexpr (kFold > 0) {
          if ((kt + u) % kFold == kFold - 1) fold();
        }
      }
    }
  }
  lin_wait<0>();  // no load outlives the workgroup
  if constexpr (kFold > 0) {
#pragma unroll
    for (int a = 0; a < TP; ++a)
#pragma unroll
      for (int b = 0; b < TQ; ++b) acc[a][b] += sum[a][b];
  }

  // acc[a][b][i]: column 4 (lane / 16) + i, row lane % 16 of its 16 x 16
  // block.  The sums go through LDS, 32 rows of every wavefront at a time, so
  // that output rows leave in whole runs and one copy of the epilogue serves
  // them all; rows are padded by 16 bytes, which spreads the lanes of a write
  // over the banks.  The barriers wait for LDS accesses alone: waiting for the
  // output's stores too, as __syncthreads does, took 19 us a tile (4096 x 1536
  // -> 4096 outputs).
  constexpr int SST = BP * 4 + 16;  // bytes of a staged row
  static_assert(WQ * 32 * SST <= NST * (OP::kBytes + OQ::kBytes), "the staged rows fit the stages");
  static_assert(TQ % 2 == 0, "two blocks of 16 rows at a time");
  char* so = lds[0];
  const long ldp = (pcols + 3) & ~3;
  const long prow0 = MODE == LIN_DW ? (long)ks_id * g.G * g.N + (long)grp * g.N : (long)ks_id * g.M;
  // A thread keeps its W columns over all rows; RS rows of a step go together.
  constexpr int W = VEC ? 4 : 2, TPR = BP / W, RPS = 64 * NW / TPR, RS = 4;
  static_assert(WQ * 32 % (RPS * RS) == 0, "whole steps of rows");
  const int cc = (threadIdx.x % TPR) * W, c = p0 + cc, r0 = threadIdx.x / TPR;
  const bool inside = c < pcols;
  float bias[W] = {};
  if constexpr (MODE == LIN_FWD) {
    if (g.bias && inside && g.splits == 1)
      load_w<ET, W, VEC>(static_cast<const ET*>(g.bias) + (long)grp * g.N + c, g.N - c, bias);
  }
  for (int b2 = 0; b2 < TQ / 2; ++b2) {
    lin_wait<63>();
    barrier();
    // (one copy of the code behind this for all blocks)
#pragma unroll
    for (int k = 0; k < TQ / 2; ++k)
      if (k == b2)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int a = 0; a < TP; ++a)
            *(f32x4*)(so + (wq * 32 + b * 16 + (lane & 15)) * SST + ((wp * TP + a) * 16 + 4 * (lane >> 4)) * 4) =
                acc[a][2 * k + b];
    lin_wait<63>();
    barrier();
    if (g.splits > 1) {
#pragma unroll 2
      for (int i = threadIdx.x; i < WQ * 32 * (BP / 4); i += 64 * NW) {
        const int sr = i / (BP / 4), c4 = 4 * (i % (BP / 4));
        const int qr = (sr >> 5) * (TQ * 16) + b2 * 32 + (sr & 31);
        if (qr < qrows && p0 + c4 < ldp)
          *(f32x4*)(g.partial + (prow0 + q0 + qr) * ldp + p0 + c4) = *(const f32x4*)(so + sr * SST + c4 * 4);
      }
      continue;
    }
    if (!inside) continue;
    auto rows = [&](auto act) QMOE_INLINE {
      for (int s0 = 0; s0 < WQ * 32; s0 += RPS * RS) {
        float z[RS][W];
        int m[RS];
        bool ok[RS];
#pragma unroll
        for (int r = 0; r < RS; ++r) {
          const int sr = s0 + r * RPS + r0;
          const int qr = (sr >> 5) * (TQ * 16) + b2 * 32 + (sr & 31);
          ok[r] = qr < qrows;
          m[r] = q0 + qr;
          const typename LinVec<float, W>::type v = *(const typename LinVec<float, W>::type*)(so + sr * SST + cc * 4);
#pragma unroll
          for (int i = 0; i < W; ++i) z[r][i] = v[i];
        }
        if constexpr (MODE == LIN_FWD) {
          linear_rows<ET, decltype(act)::value, W, RS, VEC>(g, z, bias, c, m, ok);
        } else {
          ET* out = static_cast<ET*>(g.out) + (MODE == LIN_DW ? (long)grp * g.N * g.K : 0) + c;
#pragma unroll
          for (int r = 0; r < RS; ++r)
            if (ok[r]) store_w<ET, W, VEC>(out + (long)m[r] * g.K, g.K - c, z[r]);
        }
      }
    };
    if constexpr (MODE == LIN_FWD) with_act(g.act.type, rows);
    else rows(std::integral_constant<int, kActIdentity>{});
  }
}

template <typename ET, int MODE, int BQ, int BP, int WQ, int WP, int NST>
hipError_t go_linear(const LinearGemm& g, bool vec, hipStream_t st) {
  const long rows = MODE == LIN_DW ? g.N : g.M;
  const long cols = MODE == LIN_FWD ? g.N : g.K;
  const long qb = (rows + BQ - 1) / BQ;
  const long nq = MODE == LIN_DW ? qb * g.G : g.offsets ? qb + g.G + 1 : qb;
  const long np = (cols + BP - 1) / BP;
  auto go = [&](auto v, auto t) {
    return in_launches(linear_workgroups(nq, np), [&](int b0, unsigned n) {
      const dim3 grid(n, (unsigned)g.splits), block(64 * WQ * WP);
      hipLaunchKernelGGL((qmoe_linear<ET, MODE, BQ, BP, WQ, WP, NST, decltype(v)::value, decltype(t)::value>), grid,
                         block, 0, st, g, (int)nq, (int)np, b0);
    });
  };
  auto turned = [&](auto t) { return vec ? go(std::true_type{}, t) : go(std::false_type{}, t); };
  if constexpr (MODE == LIN_FWD) {
    if (g.offsets || nq == 1) return turned(std::true_type{});
  }
  return turned(std::false_type{});
}

template <typename ET, int MODE>
hipError_t go_tile(int tile, const LinearGemm& g, hipStream_t st) {
  const bool vec = linear_vec<ET>(g, MODE);
  switch (tile) {
    case LT_256x256:
      if constexpr (sizeof(ET) == 2) return go_linear<ET, MODE, 256, 256, 2, 4, 2>(g, vec, st);
      return hipErrorInvalidValue;
    case LT_128x128: return go_linear<ET, MODE, 128, 128, 2, 2, 2>(g, vec, st);
    case LT_64x128: return go_linear<ET, MODE, 64, 128, 1, 4, 3>(g, vec, st);
    case LT_32x128: return go_linear<ET, MODE, 32, 128, 1, 4, 4>(g, vec, st);
  }
  return hipErrorInvalidValue;
}

template <typename ET>
hipError_t go_mode(int mode, int tile, const LinearGemm& g, hipStream_t st) {
  if (mode == LIN_FWD) return go_tile<ET, LIN_FWD>(tile, g, st);
  if (mode == LIN_DX) return go_tile<ET, LIN_DX>(tile, g, st);
  return go_tile<ET, LIN_DW>(tile, g, st);
}

}  // namespace qmoe
