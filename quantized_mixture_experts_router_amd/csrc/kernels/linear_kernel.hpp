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
// 32 32-bit values) or as many r rows of the other kind.
//
//  - Run-of-r tiles: row i is 8 pieces of 16 bytes, piece c in slot c ^ (i & 7)
//    (the source address is permuted, the LDS side of the load is linear), so
//    that eight lanes reading one piece of eight rows meet every bank once.
//  - The other kind, 16-bit: row r holds all BT columns; the transposing LDS
//    read gives a lane four r of its column; pieces are rotated by 64 bytes a
//    row so that the four rows of one read fall into different banks.  32-bit
//    values are read one by one.
//
// The matrix instruction's row operand is P and its column operand Q, so a
// lane ends with runs of four consecutive output columns of one output row.
#pragma once
#include <type_traits>

#include "linear_common.hpp"

namespace qmoe {

template <typename ET>
struct LinMma {  // 16-bit: 32 x 32 x 16, eight r a lane
  using Frag = typename std::conditional<std::is_same<ET, _Float16>::value, h16x8, b16x8>::type;
  static __device__ __forceinline__ f32x16 mma(Frag p, Frag q, f32x16 c) {
    if constexpr (std::is_same<ET, _Float16>::value) return __builtin_amdgcn_mfma_f32_32x32x16_f16(p, q, c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_32x32x16_bf16(p, q, c, 0, 0, 0);
  }
};
template <>
struct LinMma<float> {  // 32 x 32 x 2, four steps over the four r a lane holds
  using Frag = f32x4;
  static __device__ __forceinline__ f32x16 mma(Frag p, Frag q, f32x16 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(p[j], q[j], c, 0, 0, 0);
    return c;
  }
};

#define QMOE_LDS(p) ((__attribute__((address_space(3))) void*)(p))

// One operand's tile of BT rows or columns: fills a stage and reads fragments.
//   RUN: rows of consecutive r.  else: r rows of consecutive columns.
template <typename ET, int BT, bool RUN, int NW>
struct LinOperand {
  static constexpr int ES = sizeof(ET), EPC = 16 / ES, BK = 128 / ES;
  static constexpr int kBytes = BT * 128;              // one stage
  static constexpr int kLoads = kBytes / 1024 / NW;    // load instructions of a wavefront and stage
  static constexpr int CPR = BT * ES / 16;             // pieces per r row
  static constexpr int RPI = RUN ? 8 : 64 / CPR;       // rows one instruction covers
  static_assert(kBytes % (1024 * NW) == 0, "every wavefront issues the same count");

  const char* base;  // tile's first row or column at r = 0
  long left;         // bytes from base to the end of the operand's rows
  long step;         // bytes from stage to stage
  int ldb;           // row stride in bytes
  int voff;          // this lane's offset in an instruction's rows
  int piece;         // RUN: this lane's piece of its row

  static __device__ __forceinline__ int swz(int r) {
    if constexpr (ES == 4 || CPR < 8) return 0;  // (64-byte rows: four differ by themselves)
    if constexpr (CPR >= 16) return (r & 3) << 2;
    return ((r >> 1) & 1) << 2;  // 128-byte rows: neighbours already differ
  }

  // src: element (0, 0) of the tile; ld: row stride in elements; rows: RUN,
  // valid rows, else valid r; cols: RUN, unused, else valid columns from the
  // tile's first
  __device__ __forceinline__ void init(const ET* src, long ld, long rows, long row_len, int cols, int lane) {
    base = reinterpret_cast<const char*>(src);
    ldb = (int)(ld * ES);
    left = rows > 0 ? ((rows - 1) * ld + row_len) * ES : 0;
    if constexpr (RUN) {
      step = 128;
      piece = (lane & 7) ^ (lane >> 3);
      voff = (lane >> 3) * ldb + piece * 16;
    } else {
      step = (long)BK * ldb;
      const int r = lane / CPR;  // + a multiple of RPI: the same r & 3 (see issue)
      piece = 0;
      voff = r * ldb;
      (void)cols;
    }
  }

  // Stage kt (r from kt * BK, of R) into LDS at dst.
  __device__ __forceinline__ void issue(char* dst, long kt, long R, int cols, int wave, int lane) const {
    long rem = left - kt * step;
    rem = rem < 0 ? 0 : rem > 0x7fffffff ? 0x7fffffff : rem;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(base + kt * step), 0, (int)rem, 0x00027000);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int idx = i * NW + wave;
      int vo = voff;
      if constexpr (RUN) {
        // the last stage: pieces from R on are out of range, not the next row
        if (kt * BK + piece * EPC >= R) vo = (int)0x80000000;
      } else {
        const int r = idx * RPI + lane / CPR;
        const int c = (lane % CPR) ^ swz(r);
        vo = c * EPC < cols ? voff + c * 16 : (int)0x80000000;
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, QMOE_LDS(dst + idx * 1024), 16, vo, idx * RPI * ldb, 0, 0);
    }
  }

  // This lane's operand of k step ks (16 16-bit or 8 32-bit r) for the 32
  // rows or columns from t0 on.
  static __device__ __forceinline__ typename LinMma<ET>::Frag frag(const char* src, int t0, int ks, int lane) {
    using Frag = typename LinMma<ET>::Frag;
    if constexpr (RUN) {
      const int c = 2 * ks + (lane >> 5);
      return *(const Frag*)(src + (t0 + (lane & 31)) * 128 + ((c ^ (lane & 7)) << 4));
    } else if constexpr (ES == 4) {
      Frag f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f[j] = *(const float*)(src + (8 * ks + 4 * (lane >> 5) + j) * (BT * 4) + (t0 + (lane & 31)) * 4);
      return f;
    } else {
      union {
        s16x4 h[2];
        Frag f;
      } u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * ks + 8 * (lane >> 5) + 4 * h + ((lane & 15) >> 2);
        const int c = (t0 >> 3) + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
        u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(src + r * (BT * 2) + ((c ^ swz(r)) << 4) + (lane & 1) * 8));
      }
      return u.f;
    }
  }
};

// Output tiles are taken in runs of 32 per XCD (workgroups go to the 8 XCDs in
// turn; 32 compute units each), inside a run eight q blocks by four p blocks,
// so that a run's operand rows are shared in its XCD's L2.
__device__ __forceinline__ void tile_of(int b, int nq, int np, int& q, int& p) {
  const int t = ((b >> 3) / 32 * 8 + (b & 7)) * 32 + (b >> 3) % 32;
  const int h = min(nq, 8);
  const int s = t / (h * np), r = t - s * (h * np);
  q = s * h + r % h;
  p = r / h;
}

template <typename ET, int MODE, int BQ, int BP, int WQ, int WP, int NST, bool VEC>
__global__ void __launch_bounds__(64 * WQ * WP) qmoe_linear(const LinearGemm g, int nq, int np) {
  constexpr int NW = WQ * WP, TQ = BQ / WQ / 32, TP = BP / WP / 32;
  using OP = LinOperand<ET, BP, MODE == LIN_FWD, NW>;
  using OQ = LinOperand<ET, BQ, MODE != LIN_DW, NW>;
  constexpr int BK = OP::BK, KS = BK / (sizeof(ET) == 4 ? 8 : 16);
  __shared__ __attribute__((aligned(1024))) char lds[NST][OP::kBytes + OQ::kBytes];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  int qb, pb;
  const int ks_id = blockIdx.y;  // range of r
  tile_of(blockIdx.x, nq, np, qb, pb);
  const int p0 = pb * BP;
  int grp, lo, hi, q0, qrows;  // group, its rows from the tile on, first output row, valid rows of the tile
  const int pcols = MODE == LIN_FWD ? g.N : g.K;
  if (p0 >= pcols) return;
  OP op;
  OQ oq;
  long R;
  if constexpr (MODE == LIN_DW) {
    const int nqg = (g.N + BQ - 1) / BQ;  // q blocks of a group
    grp = qb / nqg;
    if (grp >= g.G) return;
    q0 = (qb - grp * nqg) * BQ;
    qrows = g.N - q0;
    group_rows(g.offsets, g.G, g.M, grp, lo, hi);
    R = hi - lo;
    op.init(static_cast<const ET*>(g.x) + (long)lo * g.ldx + p0, g.ldx, R, g.ldx - p0, g.K - p0, lane);
    oq.init(static_cast<const ET*>(g.dz) + (long)lo * g.lddz + q0, g.lddz, R, g.lddz - q0, g.N - q0, lane);
  } else {
    if (!find_block(g.offsets, g.G, g.M, BQ, qb, grp, lo, hi)) return;
    q0 = lo;
    qrows = hi - lo;
    if (grp == g.G && g.offsets) {  // rows behind the last group: zeros
      if (ks_id > 0 || g.splits > 1) return;  // (the finishing pass writes them)
      for (int i = threadIdx.x; i < min(qrows, BQ) * (BP / 4); i += 64 * NW) {
        const int m = q0 + i / (BP / 4), c = p0 + 4 * (i % (BP / 4));
        if constexpr (MODE == LIN_FWD) linear_zero<ET>(g, m, c);
        else store_cols4<ET, false>(static_cast<ET*>(g.out) + (long)m * g.K, c, g.K, f32x4{0.f, 0.f, 0.f, 0.f});
      }
      return;
    }
    if constexpr (MODE == LIN_FWD) {
      R = g.K;
      op.init(static_cast<const ET*>(g.w) + ((long)grp * g.N + p0) * g.ldw, g.ldw, g.N - p0, g.ldw, 0, lane);
      oq.init(static_cast<const ET*>(g.x) + (long)lo * g.ldx, g.ldx, qrows, g.ldx, 0, lane);
    } else {
      R = g.N;
      op.init(static_cast<const ET*>(g.w) + (long)grp * g.N * g.ldw + p0, g.ldw, g.N, g.ldw - p0, g.K - p0, lane);
      oq.init(static_cast<const ET*>(g.dz) + (long)lo * g.lddz, g.lddz, qrows, g.lddz, 0, lane);
    }
  }
  const int pvalid = pcols - p0;
  const long nk_all = (R + BK - 1) / BK;
  const long kb = nk_all * ks_id / g.splits, ke = nk_all * (ks_id + 1) / g.splits;
  const int nk = (int)(ke - kb);

  f32x16 acc[TP][TQ];
#pragma unroll
  for (int a = 0; a < TP; ++a)
#pragma unroll
    for (int b = 0; b < TQ; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;
  const int wq = wave / WP, wp = wave % WP;

  auto issue = [&](int kt) {
    char* dst = lds[kt % NST];
    // past the range's end: nothing is in range, the loads write zeros (the
    // count of loads in flight stays the same)
    const long k = kt < nk ? kb + kt : nk_all + kt;
    op.issue(dst, k, R, pvalid, wave, lane);
    oq.issue(dst + OP::kBytes, k, R, qrows, wave, lane);
  };
  constexpr int kInFlight = (NST - 2) * (OP::kLoads + OQ::kLoads);
#pragma unroll
  for (int s = 0; s < NST - 1; ++s) issue(s);
  for (int kt = 0; kt < nk; ++kt) {
    // stage kt has landed (this wavefront's loads; the barrier: everyone's),
    // and every wavefront has read stage kt - 1, whose place is filled next
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kInFlight) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    issue(kt + NST - 1);
    const char* sp = lds[kt % NST];
    const char* sq = sp + OP::kBytes;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      typename LinMma<ET>::Frag fp[TP], fq[TQ];
#pragma unroll
      for (int a = 0; a < TP; ++a) fp[a] = OP::frag(sp, (wp * TP + a) * 32, ks, lane);
#pragma unroll
      for (int b = 0; b < TQ; ++b) fq[b] = OQ::frag(sq, (wq * TQ + b) * 32, ks, lane);
#pragma unroll
      for (int a = 0; a < TP; ++a)
#pragma unroll
        for (int b = 0; b < TQ; ++b) acc[a][b] = LinMma<ET>::mma(fp[a], fq[b], acc[a][b]);
    }
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");  // no load outlives the workgroup

  // acc[a][b][4 j + i]: column 8 j + 4 (lane / 32) + i, row lane % 32 of its
  // 32 x 32 block.  The sums go through LDS, 32 rows of every wavefront at a
  // time, so that output rows leave in whole runs and one copy of the epilogue
  // serves them all; rows are padded by 16 bytes, which spreads the eight
  // lanes of a write over the banks.
  constexpr int SST = BP * 4 + 16;  // bytes of a staged row
  static_assert(WQ * 32 * SST <= NST * (OP::kBytes + OQ::kBytes), "the staged rows fit the stages");
  char* so = lds[0];
  const long ldp = (pcols + 3) & ~3;
  const long prow0 = MODE == LIN_DW ? (long)ks_id * g.G * g.N + (long)grp * g.N : (long)ks_id * g.M;
#pragma unroll
  for (int b = 0; b < TQ; ++b) {
    __syncthreads();
#pragma unroll
    for (int a = 0; a < TP; ++a)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *(f32x4*)(so + (wq * 32 + (lane & 31)) * SST + ((wp * TP + a) * 32 + 8 * j + 4 * (lane >> 5)) * 4) =
            f32x4{acc[a][b][4 * j], acc[a][b][4 * j + 1], acc[a][b][4 * j + 2], acc[a][b][4 * j + 3]};
    __syncthreads();
#pragma unroll 2
    for (int i = threadIdx.x; i < WQ * 32 * (BP / 4); i += 64 * NW) {
      const int sr = i / (BP / 4), cc = 4 * (i % (BP / 4));
      const int qr = ((sr >> 5) * TQ + b) * 32 + (sr & 31);
      if (qr >= qrows) continue;
      const f32x4 v = *(const f32x4*)(so + sr * SST + cc * 4);
      const int m = q0 + qr, c = p0 + cc;
      if (g.splits > 1) {
        if (c < ldp) *(f32x4*)(g.partial + (prow0 + m) * ldp + c) = v;
      } else if constexpr (MODE == LIN_FWD) {
        linear_epilogue<ET, VEC>(g, grp, m, c, v);
      } else {
        ET* row = static_cast<ET*>(g.out) + (MODE == LIN_DW ? ((long)grp * g.N + m) * g.K : (long)m * g.K);
        store_cols4<ET, VEC>(row, c, g.K, v);
      }
    }
  }
}

template <typename ET, int MODE, int BQ, int BP, int WQ, int WP, int NST>
hipError_t go_linear(const LinearGemm& g, bool vec, hipStream_t st) {
  const long rows = MODE == LIN_DW ? g.N : g.M;
  const long cols = MODE == LIN_FWD ? g.N : g.K;
  const long qb = (rows + BQ - 1) / BQ;
  const long nq = MODE == LIN_DW ? qb * g.G : g.offsets ? qb + g.G + 1 : qb;
  const long np = (cols + BP - 1) / BP;
  const long h = nq < 8 ? nq : 8;
  const long n = (nq + h - 1) / h * h * np;  // whole runs of h q blocks
  const dim3 grid((unsigned)((n + 255) / 256 * 256), (unsigned)g.splits), block(64 * WQ * WP);
  if (vec) hipLaunchKernelGGL((qmoe_linear<ET, MODE, BQ, BP, WQ, WP, NST, true>), grid, block, 0, st, g, (int)nq, (int)np);
  else hipLaunchKernelGGL((qmoe_linear<ET, MODE, BQ, BP, WQ, WP, NST, false>), grid, block, 0, st, g, (int)nq, (int)np);
  return hipGetLastError();
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
