// Routing weights, tokens sorted by expert and back, each with its gradient:
// launch functions (host side; enqueue only).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace qmoe {

enum RowType { ROW_F32 = 0, ROW_F16 = 1, ROW_BF16 = 2 };

// k largest logits of each row (idx, -1 where masked experts are all that is
// left) and their softmax weights, over the selection or (over_all) over
// every expert.
hipError_t launch_route_topk(const float* logits, int T, int E, int k, bool over_all, int* idx, float* w,
                             hipStream_t st);
hipError_t launch_route_grad(const float* gw, const float* logits, const void* idx, bool idx64, int T, int E, int k,
                             bool over_all, float* gl, hipStream_t st);

// Slots per block of the expert sort.  Up to kSortSelf slots every block
// counts the experts of all slots itself; beyond, a first launch counts per
// block, with at most 256 blocks (each adds up the others').  One launch against
// two, us: 4096 slots 4.6 / 7.4 (8 experts) and 5.0 / 8.8 (256), 12288 slots
// 6.3 / 7.9 and 6.3 / 9.6, 16384 slots 7.1 / 7.6 and 6.9 / 8.7, 24576 slots
// 8.9 / 8.1 and 8.2 / 9.2, 32768 slots 10.6 / 8.9 and 9.5 / 9.8.
constexpr int kSortRound = 512;
constexpr int kSortSelf = 16384;
inline int sort_chunk(long S) {
  if (S <= kSortSelf) return kSortRound;
  const long c = std::max((S + 255) / 256, 1024l);
  return (int)((c + kSortRound - 1) / kSortRound * kSortRound);
}
// Stable sort of the S slots by expert: offsets [E + 1], perm [S] (may be
// NULL), inverse [S] (place, or -1 - place of a slot whose index lies outside
// [0, E): those follow the last expert, in slot order).  hist: blocks x
// (E + 1) ints beyond kSortSelf slots.
hipError_t launch_sort_slots(const void* idx, bool idx64, int S, int E, int* hist, int* offsets, int* perm,
                             int* inverse, hipStream_t st);

// Rows of H elements.  dispatch: rows[place of (t, s)] = x[t], zeros at the
// places of dropped slots.
hipError_t launch_dispatch_rows(int type, const void* x, const int* inverse, int T, int k, long H, void* rows,
                                hipStream_t st);
// out[t] = sum_s w[t, s] rows[inverse[t, s]] (w NULL: 1), slots in order,
// dropped ones and places outside [0, T k) left out.
hipError_t launch_combine_rows(int type, const void* rows, const int* inverse, const float* w, int T, int k, long H,
                               void* out, hipStream_t st);
// grows[inverse[t, s]] = w[t, s] gout[t], gw[t, s] = <gout[t], rows[inverse[t, s]]>; zeros for dropped slots.
// grows or gw may be NULL.
hipError_t launch_combine_grad(int type, const void* gout, const void* rows, const int* inverse, const float* w,
                               int T, int k, long H, void* grows, float* gw, hipStream_t st);

}  // namespace qmoe
