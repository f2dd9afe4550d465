// Routing weights from logits, tokens sorted by expert and back, each with its
// gradient (tokens.h).
//
// Everything here is bound by HBM (rows) or by launch latency (small calls):
// rows move 16 bytes a lane, a row that several slots share is read once
// (dispatch) and a row's sum stays in registers (combine), with no atomics:
// every output element has one writer, so results do not depend on order.
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "launches.h"
#include "tokens.h"

namespace qmoe {

namespace {

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

__device__ __forceinline__ int read_index(const void* idx, bool idx64, long i) {
  if (!idx64) return static_cast<const int*>(idx)[i];
  const int64_t v = static_cast<const int64_t*>(idx)[i];
  return (v < 0 || v > 0x7fffffff) ? -1 : (int)v;
}

// One wavefront per token, logits e = lane + 64 j in registers.  A round takes
// the largest value left (one wavefront maximum), then the lowest expert that
// holds it (a ballot per register).  Bound by launch latency in decode (16 x 8
// logits: 2.5 us).
template <int V>
__global__ void __launch_bounds__(256) qmoe_route_topk(const float* __restrict__ logits, int T, int E, int k,
                                                       bool over_all, int b0, int* __restrict__ idx,
                                                       float* __restrict__ w) {
  const int t = (b0 + blockIdx.x) * 4 + (threadIdx.x >> 6), lane = lane_id();
  if (t >= T) return;
  const float* row = logits + (long)t * E;
  float v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float x = lane + 64 * j < E ? row[lane + 64 * j] : -INFINITY;
    v[j] = x != x ? -INFINITY : x;
  }
  float top = 0.f, sum = 0.f;
  if (over_all) {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, v[j]);
    top = wave_max(m);
    top = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int j = 0; j < V; ++j) sum += expf(v[j] - top);
    sum = wave_sum(sum);
  }
  // pick r waits in lane r % 64 of register r / 64: written out below
  float pv[V];
  int pe[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    pv[j] = 0.f;
    pe[j] = -1;
  }
  for (int r = 0; r < k; ++r) {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, v[j]);
    m = wave_max(m);
    if (m == -INFINITY) break;  // only masked experts are left
    int e = -1;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const unsigned long long b = __ballot(v[j] == m);
      if (e < 0 && b) {
        const int l = __ffsll((long long)b) - 1;
        e = l + 64 * j;
        if (lane == l) v[j] = -INFINITY;
      }
    }
    if (!over_all) {
      if (r == 0) top = m;
      sum += expf(m - top);
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (r == lane + 64 * j) {
        pv[j] = expf(m - top);
        pe[j] = e;
      }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int r = lane + 64 * j;
    if (r < k) {
      idx[(long)t * k + r] = pe[j];
      w[(long)t * k + r] = pe[j] < 0 ? 0.f : pv[j] / sum;
    }
  }
}

// One wavefront per token.  With w the weights and mean = sum_s w_s g_s:
//   softmax over the selection:  gl[e] = sum over slots s of e of w_s (g_s - mean)
//   softmax over all experts:    gl[e] = (the same of w_s g_s) - p_e mean
// A lane adds up its experts' slots in slot order (no atomics, and the same
// expert twice adds twice).  8192 x 128 logits, k = 8: 6.7 us against 1.8 us of
// bytes; the chain index -> logit -> sums of a token and the k slots' LDS reads
// bound it.
template <int V>
__global__ void __launch_bounds__(256) qmoe_route_grad(const float* __restrict__ gw, const float* __restrict__ logits,
                                                       const void* __restrict__ idx, bool idx64, int T, int E, int k,
                                                       bool over_all, int b0, float* __restrict__ gl) {
  extern __shared__ char smem[];  // per wavefront: k experts, k values
  const int wave = threadIdx.x >> 6, lane = lane_id();
  int* se = reinterpret_cast<int*>(smem) + wave * 2 * k;
  float* sv = reinterpret_cast<float*>(se + k);
  const int t = (b0 + blockIdx.x) * 4 + wave;
  if (t >= T) return;
  const float* row = logits + (long)t * E;
  float v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float x = lane + 64 * j < E ? row[lane + 64 * j] : -INFINITY;
    v[j] = x != x ? -INFINITY : x;
  }
  // each lane handles slots lane, lane + 64, ...: expert and logit into LDS
  float top = -INFINITY, sum = 0.f;
  for (int s = lane; s < k; s += 64) {
    int e = read_index(idx, idx64, (long)t * k + s);
    float x = -INFINITY;
    if (e >= 0 && e < E) {
      x = row[e];
      x = x != x ? -INFINITY : x;
    }
    if (x == -INFINITY) e = -1;  // masked: weight 0
    se[s] = e;
    sv[s] = x;
    top = fmaxf(top, x);
  }
  if (over_all) {
#pragma unroll
    for (int j = 0; j < V; ++j) top = fmaxf(top, v[j]);
  }
  top = wave_max(top);
  if (top == -INFINITY) top = 0.f;
  if (over_all) {
#pragma unroll
    for (int j = 0; j < V; ++j) sum += expf(v[j] - top);
  } else {
    for (int s = lane; s < k; s += 64) sum += expf(sv[s] - top);
  }
  sum = wave_sum(sum);
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  float mean = 0.f;
  for (int s = lane; s < k; s += 64) {
    const float ws = se[s] < 0 ? 0.f : expf(sv[s] - top) * inv;
    const float a = ws == 0.f ? 0.f : ws * gw[(long)t * k + s];
    mean += a;
    sv[s] = over_all ? a : ws;
  }
  mean = wave_sum(mean);
  if (!over_all)
    for (int s = lane; s < k; s += 64) sv[s] = se[s] < 0 ? 0.f : sv[s] * (gw[(long)t * k + s] - mean);
  // (one wavefront's own LDS words: written and read in program order)
  __builtin_amdgcn_wave_barrier();
  float out[V];
#pragma unroll
  for (int j = 0; j < V; ++j) out[j] = over_all ? -expf(v[j] - top) * inv * mean : 0.f;
  for (int s = 0; s < k; ++s) {
    const int e = se[s];
    const float a = sv[s];
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (e == lane + 64 * j) out[j] += a;
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (lane + 64 * j < E) gl[(long)t * E + lane + 64 * j] = out[j];
}

// ------------------------------------------------------------------ sort
// Expert bucket of a slot: E collects the indices outside [0, E).
__device__ __forceinline__ int bucket(const void* idx, bool idx64, int s, int E) {
  const int e = read_index(idx, idx64, s);
  return (e < 0 || e >= E) ? E : e;
}

__global__ void __launch_bounds__(kSortRound) qmoe_sort_count(const void* __restrict__ idx, bool idx64, int S, int E,
                                                              int chunk, int* __restrict__ hist) {
  extern __shared__ int cnt[];  // [E + 1]
  for (int e = threadIdx.x; e <= E; e += kSortRound) cnt[e] = 0;
  __syncthreads();
  const int s1 = min(S, (int)(blockIdx.x + 1) * chunk);
  for (int s = blockIdx.x * chunk + threadIdx.x; s < s1; s += kSortRound)
    atomicAdd(&cnt[bucket(idx, idx64, s, E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kSortRound) hist[(long)blockIdx.x * (E + 1) + e] = cnt[e];
}

// Places of a chunk's slots.  The block adds up the chunks' counts itself
// (first place of every expert in this chunk; hist NULL: it counts them from
// the indices), then ranks 512 slots a round: lanes of one wavefront with the
// same expert find each other with a ballot per bit of the expert's number,
// wavefronts in order through LDS counts.
// Bound by latency: 12288 slots of 64 experts take 7.2 us (11.4 us with four
// loads in flight a thread and a second count of what comes before the chunk).
__global__ void __launch_bounds__(kSortRound) qmoe_sort_place(const void* __restrict__ idx, bool idx64, int S, int E,
                                                              int chunk, int nchunks, const int* __restrict__ hist,
                                                              int* __restrict__ offsets, int* __restrict__ perm,
                                                              int* __restrict__ inverse) {
  constexpr int NW = kSortRound / 64;
  extern __shared__ int sm[];
  const int B = E + 1;
  int* base = sm;          // [B] next place of every bucket
  int* wcnt = sm + B;      // [NW][B] counts of a round's wavefronts
  __shared__ int wsum[NW];
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int s0 = blockIdx.x * chunk, s1 = min(S, s0 + chunk);
  const int e0 = s0 + (int)threadIdx.x < s1 ? bucket(idx, idx64, s0 + threadIdx.x, E) : 0;
  if (!hist) {
    for (int e = threadIdx.x; e < 2 * B; e += kSortRound) sm[e] = 0;
    __syncthreads();
    // (what comes before the chunk in wcnt, the rest in base; eight indices
    // in flight a thread)
    for (int s = threadIdx.x; s < S; s += 8 * kSortRound) {
      int e[8];
      if (idx64) {
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = bucket(idx, true, min(s + j * kSortRound, S - 1), E);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = bucket(idx, false, min(s + j * kSortRound, S - 1), E);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = s + j * kSortRound;
        if (at < S) atomicAdd(&(at < s0 ? wcnt : base)[e[j]], 1);
      }
    }
    __syncthreads();
  }
  // totals of buckets 2 i and 2 i + 1 in thread i (B <= 1024), and this
  // chunk's own start among them
  int tot[2] = {0, 0}, before[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = 2 * threadIdx.x + h;
    if (e >= B) continue;
    if (!hist) {
      before[h] = wcnt[e];
      tot[h] = base[e] + before[h];
    } else {
#pragma unroll 8
      for (int c = 0; c < nchunks; ++c) {
        const int n = hist[(long)c * B + e];
        tot[h] += n;
        before[h] += c < (int)blockIdx.x ? n : 0;
      }
    }
  }
  int inc = tot[0] + tot[1];
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  int first = inc - tot[0] - tot[1];
  for (int i = 0; i < wave; ++i) first += wsum[i];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = 2 * threadIdx.x + h;
    if (e < B) {
      const int f = first + (h ? tot[0] : 0);
      base[e] = f + before[h];
      if (blockIdx.x == 0) offsets[e] = f;  // e == E: the first place behind the last expert
    }
  }
  int bits = 0;
  while ((1 << bits) < B) ++bits;
  for (int r0 = s0; r0 < s1; r0 += kSortRound) {
    for (int i = threadIdx.x; i < NW * B; i += kSortRound) wcnt[i] = 0;
    __syncthreads();
    const int s = r0 + threadIdx.x;
    const bool valid = s < s1;
    const int e = r0 == s0 ? e0 : valid ? bucket(idx, idx64, s, E) : 0;
    unsigned long long same = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
      const unsigned long long m = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1ull));
    if (valid && rank == 0) wcnt[wave * B + e] = __popcll(same);
    __syncthreads();
    if (valid) {
      int at = base[e] + rank;
      for (int i = 0; i < wave; ++i) at += wcnt[i * B + e];
      if (perm) perm[at] = s;
      inverse[s] = e < E ? at : -1 - at;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < B; i += kSortRound) {
      int add = 0;
#pragma unroll
      for (int j = 0; j < NW; ++j) add += wcnt[j * B + i];
      base[i] += add;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ rows
// A piece of a row: 16 bytes (whole rows of such pieces) or one element.
template <typename ET, bool WIDE>
struct Piece {
  static constexpr int N = WIDE ? 16 / sizeof(ET) : 1;
  typedef ET type __attribute__((ext_vector_type(N)));
};
template <typename ET>
struct Piece<ET, false> {
  static constexpr int N = 1;
  typedef ET type;
};
template <typename ET, bool WIDE>
__device__ __forceinline__ float piece_at(const typename Piece<ET, WIDE>::type& p, int i) {
  if constexpr (WIDE) return (float)p[i];
  else return (float)p;
}
template <typename ET, bool WIDE>
__device__ __forceinline__ void piece_set(typename Piece<ET, WIDE>::type& p, int i, float v) {
  if constexpr (WIDE) p[i] = (ET)v;
  else p = (ET)v;
}

// A thread per piece of a token's row: `per` threads a token (a power of two
// up to 256), the rest of the row in blockIdx.y.  Bound by HBM: 2048 rows of 4 KB
// to 6 places each (59 MB) in 10.4 us, 5.6 TB/s.
template <typename U>
__global__ void __launch_bounds__(256) qmoe_dispatch_rows(const U* __restrict__ x, const int* __restrict__ inverse,
                                                          int T, int k, long pieces, int per_log, int b0,
                                                          U* __restrict__ rows) {
  const long t = ((long)(b0 + blockIdx.x) << (8 - per_log)) + (threadIdx.x >> per_log);
  const long c = ((long)blockIdx.y << per_log) + (threadIdx.x & ((1 << per_log) - 1));
  if (t >= T || c >= pieces) return;
  const U v = x[t * pieces + c];
  const int* inv = inverse + t * k;
  for (int s = 0; s < k; ++s) {
    const int p = inv[s];
    rows[(long)(p < 0 ? -1 - p : p) * pieces + c] = p < 0 ? U{} : v;
  }
}

// A token's sum in registers, four of its rows in flight at a time, `per`
// threads a token as above.  Bound by HBM: 65536 rows of 8 KB, half of them
// dropped, to 8192 sums (278 MB to move) in 67 us, 4.1 TB/s.
template <typename ET, bool WIDE>
__global__ void __launch_bounds__(256) qmoe_combine_rows(const ET* __restrict__ rows, const int* __restrict__ inverse,
                                                         const float* __restrict__ w, int T, int k, long pieces,
                                                         int per_log, int b0, ET* __restrict__ out) {
  using P = Piece<ET, WIDE>;
  using V = typename P::type;
  const long t = ((long)(b0 + blockIdx.x) << (8 - per_log)) + (threadIdx.x >> per_log);
  const long c = ((long)blockIdx.y << per_log) + (threadIdx.x & ((1 << per_log) - 1));
  if (t >= T || c >= pieces) return;
  const V* src = reinterpret_cast<const V*>(rows) + c;
  const int S = T * k;
  float acc[P::N];
#pragma unroll
  for (int i = 0; i < P::N; ++i) acc[i] = 0.f;
  for (int s0 = 0; s0 < k; s0 += 4) {
    // four rows in flight; a dropped slot reads row 0 and adds nothing
    V v[4];
    float f[4];
    bool use[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p = s0 + j < k ? inverse[t * k + s0 + j] : -1;
      use[j] = p >= 0 && p < S;
      f[j] = use[j] && w ? w[t * k + s0 + j] : 1.f;
      v[j] = src[(use[j] ? (long)p : 0) * pieces];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < P::N; ++i)
        acc[i] = use[j] ? fmaf(f[j], piece_at<ET, WIDE>(v[j], i), acc[i]) : acc[i];
  }
  V o;
#pragma unroll
  for (int i = 0; i < P::N; ++i) piece_set<ET, WIDE>(o, i, acc[i]);
  reinterpret_cast<V*>(out)[t * pieces + c] = o;
}

// A wavefront per slot (the slots of one token are neighbours and share its
// gradient row in the caches): the row's product with its weight, and the dot
// product, 64 pieces a step, added up across the wavefront at the end.  Bound by
// HBM: 12282 rows of 4 KB read and written (109 MB) in 19.7 us, 5.5 TB/s.
template <typename ET, bool WIDE>
__global__ void __launch_bounds__(256) qmoe_combine_grad(const ET* __restrict__ gout, const ET* __restrict__ rows,
                                                         const int* __restrict__ inverse, const float* __restrict__ w,
                                                         int S, int k, long pieces, int b0, ET* __restrict__ grows,
                                                         float* __restrict__ gw) {
  using P = Piece<ET, WIDE>;
  using V = typename P::type;
  const long s = (long)(b0 + blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (s >= S) return;
  const int lane = lane_id();
  const int p = inverse[s];
  const bool held = p >= 0;
  const int at = held ? p : -1 - p;
  if (at >= S) {  // not a place
    if (gw && lane == 0) gw[s] = 0.f;
    return;
  }
  const V* g = reinterpret_cast<const V*>(gout) + s / k * pieces;
  const V* r = reinterpret_cast<const V*>(rows) + at * pieces;
  V* o = reinterpret_cast<V*>(grows) + at * pieces;
  const float ws = w[s];
  float dot = 0.f;
  if (!held) {
    if (grows)
      for (long c = lane; c < pieces; c += 64) o[c] = V{};
  } else {
#pragma unroll 2
    for (long c = lane; c < pieces; c += 64) {
      const V a = g[c];
      if (gw) {
        const V b = r[c];
#pragma unroll
        for (int i = 0; i < P::N; ++i) dot = fmaf(piece_at<ET, WIDE>(a, i), piece_at<ET, WIDE>(b, i), dot);
      }
      if (grows) {
        V v;
#pragma unroll
        for (int i = 0; i < P::N; ++i) piece_set<ET, WIDE>(v, i, ws * piece_at<ET, WIDE>(a, i));
        o[c] = v;
      }
    }
  }
  if (gw) {
    dot = wave_sum(dot);
    if (lane == 0) gw[s] = dot;
  }
}

bool wide_ok(long row_bytes, std::initializer_list<const void*> ps) {
  if (row_bytes % 16) return false;
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 15) return false;
  return true;
}

// Threads a token (log2) and the grid for rows of `pieces`: workgroups of
// tokens in x, of pieces in y.
struct RowGrid {
  int per_log;
  long x;
  unsigned y;
};
RowGrid row_grid(long T, long pieces) {
  int l = 0;
  while (l < 8 && (1l << l) < pieces) ++l;
  const long tb = 1l << (8 - l);
  return {l, (T + tb - 1) / tb, (unsigned)((pieces + (1l << l) - 1) >> l)};
}

template <typename ET>
hipError_t combine_rows_t(const void* rows, const int* inverse, const float* w, int T, int k, long H, void* out,
                          hipStream_t st) {
  const bool wide = wide_ok(H * (long)sizeof(ET), {rows, out});
  const long pieces = wide ? H * (long)sizeof(ET) / 16 : H;
  const RowGrid r = row_grid(T, pieces);
  return in_launches(r.x, [&](int b0, unsigned n) {
    const dim3 grid(n, r.y), block(256);
    if (wide)
      hipLaunchKernelGGL((qmoe_combine_rows<ET, true>), grid, block, 0, st, (const ET*)rows, inverse, w, T, k, pieces, r.per_log, b0, (ET*)out);
    else
      hipLaunchKernelGGL((qmoe_combine_rows<ET, false>), grid, block, 0, st, (const ET*)rows, inverse, w, T, k, pieces, r.per_log, b0, (ET*)out);
  });
}

template <typename ET>
hipError_t combine_grad_t(const void* gout, const void* rows, const int* inverse, const float* w, int T, int k, long H,
                          void* grows, float* gw, hipStream_t st) {
  const bool wide = wide_ok(H * (long)sizeof(ET), {gout, rows, grows});
  const long pieces = wide ? H * (long)sizeof(ET) / 16 : H;
  const int S = T * k;
  return in_launches((S + 3) / 4, [&](int b0, unsigned n) {
    const dim3 grid(n), block(256);
    if (wide)
      hipLaunchKernelGGL((qmoe_combine_grad<ET, true>), grid, block, 0, st, (const ET*)gout, (const ET*)rows, inverse, w, S, k, pieces, b0, (ET*)grows, gw);
    else
      hipLaunchKernelGGL((qmoe_combine_grad<ET, false>), grid, block, 0, st, (const ET*)gout, (const ET*)rows, inverse, w, S, k, pieces, b0, (ET*)grows, gw);
  });
}

}  // namespace

// ---------------------------------------------------------------- launchers
#define QMOE_BY_REGS(CALL)                                  \
  {                                                         \
    const int v_ = (E + 63) / 64;                           \
    if (v_ <= 1) CALL(1);                                   \
    else if (v_ <= 2) CALL(2);                              \
    else if (v_ <= 4) CALL(4);                              \
    else if (v_ <= 8) CALL(8);                              \
    else CALL(16);                                          \
  }

hipError_t launch_route_topk(const float* logits, int T, int E, int k, bool over_all, int* idx, float* w,
                             hipStream_t st) {
  return in_launches((T + 3) / 4, [&](int b0, unsigned n) {
    const dim3 grid(n), block(256);
#define QMOE_CALL(VV) \
  hipLaunchKernelGGL(qmoe_route_topk<VV>, grid, block, 0, st, logits, T, E, k, over_all, b0, idx, w)
    QMOE_BY_REGS(QMOE_CALL)
#undef QMOE_CALL
  });
}

hipError_t launch_route_grad(const float* gw, const float* logits, const void* idx, bool idx64, int T, int E, int k,
                             bool over_all, float* gl, hipStream_t st) {
  const size_t lds = (size_t)4 * 2 * k * 4;
  return in_launches((T + 3) / 4, [&](int b0, unsigned n) {
    const dim3 grid(n), block(256);
#define QMOE_CALL(VV) \
  hipLaunchKernelGGL(qmoe_route_grad<VV>, grid, block, lds, st, gw, logits, idx, idx64, T, E, k, over_all, b0, gl)
    QMOE_BY_REGS(QMOE_CALL)
#undef QMOE_CALL
  });
}

hipError_t launch_sort_slots(const void* idx, bool idx64, int S, int E, int* hist, int* offsets, int* perm,
                             int* inverse, hipStream_t st) {
  const int chunk = sort_chunk(S), n = S > 0 ? (S + chunk - 1) / chunk : 1;
  const size_t B = E + 1;
  if (S <= kSortSelf) hist = nullptr;
  else
    hipLaunchKernelGGL(qmoe_sort_count, dim3(n), dim3(kSortRound), B * sizeof(int), st, idx, idx64, S, E, chunk, hist);
  hipLaunchKernelGGL(qmoe_sort_place, dim3(n), dim3(kSortRound), (1 + kSortRound / 64) * B * sizeof(int), st, idx,
                     idx64, S, E, chunk, n, hist, offsets, perm, inverse);
  return hipGetLastError();
}

hipError_t launch_dispatch_rows(int type, const void* x, const int* inverse, int T, int k, long H, void* rows,
                                hipStream_t st) {
  const long es = type == ROW_F32 ? 4 : 2;
  const bool wide = wide_ok(H * es, {x, rows});
  const long pieces = wide ? H * es / 16 : H;
  const RowGrid r = row_grid(T, pieces);
  return in_launches(r.x, [&](int b0, unsigned n) {
    const dim3 grid(n, r.y), block(256);
    if (wide)
      hipLaunchKernelGGL(qmoe_dispatch_rows<u32x4>, grid, block, 0, st, (const u32x4*)x, inverse, T, k, pieces, r.per_log, b0, (u32x4*)rows);
    else if (es == 4)
      hipLaunchKernelGGL(qmoe_dispatch_rows<uint32_t>, grid, block, 0, st, (const uint32_t*)x, inverse, T, k, pieces, r.per_log, b0, (uint32_t*)rows);
    else
      hipLaunchKernelGGL(qmoe_dispatch_rows<uint16_t>, grid, block, 0, st, (const uint16_t*)x, inverse, T, k, pieces, r.per_log, b0, (uint16_t*)rows);
  });
}

hipError_t launch_combine_rows(int type, const void* rows, const int* inverse, const float* w, int T, int k, long H,
                               void* out, hipStream_t st) {
  if (type == ROW_F32) return combine_rows_t<float>(rows, inverse, w, T, k, H, out, st);
  if (type == ROW_F16) return combine_rows_t<_Float16>(rows, inverse, w, T, k, H, out, st);
  return combine_rows_t<__bf16>(rows, inverse, w, T, k, H, out, st);
}

hipError_t launch_combine_grad(int type, const void* gout, const void* rows, const int* inverse, const float* w,
                               int T, int k, long H, void* grows, float* gw, hipStream_t st) {
  if (type == ROW_F32) return combine_grad_t<float>(gout, rows, inverse, w, T, k, H, grows, gw, st);
  if (type == ROW_F16) return combine_grad_t<_Float16>(gout, rows, inverse, w, T, k, H, grows, gw, st);
  return combine_grad_t<__bf16>(gout, rows, inverse, w, T, k, H, grows, gw, st);
}

}  // namespace qmoe
