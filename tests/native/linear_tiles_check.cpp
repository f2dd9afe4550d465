// The order of the linear layers' tiles (csrc/kernels/linear_tiles.h) on the
// host: every tile of nq x np comes up once, for the launch of exactly nq q
// blocks and for the larger launches of a bound on them, and at the limits of
// the contract no product leaves 32 bits (undefined-behaviour sanitizer).
#include <cstdio>
#include <vector>

#include "kernels/linear_tiles.h"

using namespace qmoe;

static long failures = 0;

static void cover(int nq, int np, int bound) {
  const long wg = linear_workgroups(bound, np);
  std::vector<int> seen((size_t)nq * np, 0);
  for (long b = 0; b < wg; ++b) {
    const LinearTileAt t = linear_tile_of((int)b, nq, np);
    if (t.q < 0 || t.p < 0) ++failures;
    else if (t.q < nq && t.p < np) ++seen[(size_t)t.q * np + t.p];
  }
  for (int n : seen) failures += n != 1;
}

int main() {
  long cases = 0;
  for (int nq = 1; nq <= 40; ++nq)
    for (int np = 1; np <= 40; ++np)
      for (int more : {0, 1, 7, 9, 33, 200}) cover(nq, np, nq + more), ++cases;
  for (int nq : {63, 64, 65, 127, 500, 1000})
    for (int np : {1, 2, 7, 8, 12, 31, 64, 229})
      for (int more : {0, 1, 17, 1023}) cover(nq, np, nq + more), ++cases;
  // the most tiles that the contract admits: nq (np + 1) below 2^31 - 512 with room for eight more q blocks
  const long most = (1L << 31) - 513;
  for (long np = 1; np <= 8192; np = np * 2 + (np % 3)) {
    const long nq = most / (np + 1) - 9;
    const long wg = linear_workgroups(nq, np);
    for (long b : {0L, 1L, wg / 2, wg - 1}) {
      if (b >= (1L << 31)) continue;
      const LinearTileAt t = linear_tile_of((int)b, (int)nq, (int)np);
      failures += t.q < 0 || t.p < 0 || t.p > np + 8;
      ++cases;
    }
  }
  std::printf("%ld cases, %ld failures\n", cases, failures);
  return failures != 0;
}
