// The order of the linear layers' output tiles over the workgroups of a launch
// (plain C++: the kernel and the host share it).
#pragma once

namespace qmoe {

struct LinearTileAt {
  int q, p;
};

// Output tiles are taken in runs of up to 32 per XCD (workgroups go to the 8
// XCDs in turn; 32 compute units each; every XCD gets the same number of runs),
// inside a run eight q blocks by four p blocks, so that a run's operand rows
// are shared in its XCD's L2.  Tile of workgroup b of nq x np tiles, both at
// least 1; some b's tiles lie past nq or np.
constexpr LinearTileAt linear_tile_of(int b, int nq, int np) {
  const int h = nq < 8 ? nq : 8;
  const int share = ((nq + h - 1) / h * h * np + 7) >> 3, runs = (share + 31) >> 5, run = (share + runs - 1) / runs;
  const int t = ((b >> 3) / run * 8 + (b & 7)) * run + (b >> 3) % run;
  const int s = t / (h * np), r = t - s * (h * np);
  return {s * h + r % h, r / h};
}

// Workgroups that cover nq x np tiles, or fewer q blocks of as many p blocks.
constexpr long linear_workgroups(long nq, long np) {
  const long h = nq < 8 ? nq : 8;
  if (h <= 0 || np <= 0) return 0;
  const long share = ((nq + h - 1) / h * h * np + 7) / 8;
  return (share <= 32 ? share : (share + 31) / 32 * 32) * 8;
}

}  // namespace qmoe
