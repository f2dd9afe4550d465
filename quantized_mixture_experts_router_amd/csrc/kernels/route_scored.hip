// Routing from scores (route_scored.h).
#include <math.h>

#include "common.hpp"
#include "launches.h"
#include "route_scored.h"
#include "wave.hpp"

namespace qmoe {

namespace {

// Signed integers that order like the floats (which are not NaN and no -0).
__device__ __forceinline__ int key_of(float v) {
  const int b = __float_as_int(v);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float of_key(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }
constexpr int kNone = (int)0x807fffff;  // -infinity

// Register j of a lane holds element lane + 64 j of a row of E; `none` past its end.
template <int V>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane, float none, float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane + 64 * j;
    v[j] = row[min(e, E - 1)];  // (no branch: the loads go out together)
  }
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = lane + 64 * j < E ? v[j] : none;
}
// A row's logits: +infinity counts as the largest float, -infinity and NaN
// (masked) come back as -infinity.
template <int V>
__device__ __forceinline__ void load_logits(const float* __restrict__ row, int E, int lane, float (&v)[V]) {
  load_row<V>(row, E, lane, -INFINITY, v);
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = fminf(fmaxf(v[j], -INFINITY), 3.4028234664e38f);  // (the larger of NaN and a number is the number)
}

// x[j] <- e^x[j] for x in [-110, 0] in 64 bits, within 2^-50 of itself (the
// polynomial of degree 10 through e^r at the Chebyshev points of |r| <= ln 2 / 2).
template <int V>
__device__ __forceinline__ void exp_below(double (&x)[V]) {
  constexpr double c[] = {2.764019739169484e-06, 2.480150431378554e-05, 0.00019841170230570286, 0.001388888893251478,
                          0.008333333385699212,  0.041666666666573066,  0.16666666666554314,    0.5000000000000006,
                          1.0000000000000067,    1.0};
  double n[V], p[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    n[j] = __builtin_rint(x[j] * 1.4426950408889634);
    x[j] = fma(n[j], -0.6931471805599453, x[j]);
    x[j] = fma(n[j], -2.3190468138462996e-17, x[j]);
    p[j] = 2.762637106569636e-07;
  }
#pragma unroll
  for (int i = 0; i < 10; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = fma(p[j], x[j], c[i]);
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = __builtin_ldexp(p[j], (int)n[j]);
}
// 1 / d for normal d, within 2^-51 of itself: the hardware's estimate (2^-23 at least) and two steps of Newton's method.
__device__ __forceinline__ double reciprocal(double d) {
  double y = __builtin_amdgcn_rcp(d);
  y = fma(y, fma(-d, y, 1.0), y);
  return fma(y, fma(-d, y, 1.0), y);
}

// One wavefront per token, expert lane + 64 j in register j.  The scores are
// evaluated in 64 bits and rounded once to float32: an expert is selected by
// comparing its score plus bias with others', and two that differ in float32's
// last bits would change places with the rounding errors of a float32 exponential.
//
// Bound by the vector instructions (524 a wavefront below, a fifth of them the 64-bit
// exponentials; their issue counts 14.6 us of SIMD time if the clock is 2.4 GHz, which
// was not measured): reductions stay in registers, ranks of groups
// are counted by all lanes, and a round of the selection is one reduction, a compare
// a register (whose ballots give the lowest expert that holds the largest key) and
// a write to one lane.  16384 x 256 logits, 6 out of 5 of 16 groups, softmax: 17.0
// us in a row of calls, 19.0 traced alone (30.5 with reductions and scores through
// LDS and library exponentials) where its bytes take 3.4; 8 out of 4 of 8 groups,
// sigmoid: 18.5 us; 16 x 128, sigmoid: 4.1 us.
// k <= 64 (else MANY: pick r in lane r % 64 of register r / 64).
template <int V, bool MANY>
__global__ void __launch_bounds__(256) qmoe_route_scored(const float* __restrict__ logits,
                                                         const float* __restrict__ bias, int T, RouteScored a, int b0,
                                                         int* __restrict__ idx, float* __restrict__ w) {
  __shared__ int lds[4][64 * V];  // per wavefront: ranks, then groups' ranks, then the scores' bits
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  const int t = (b0 + blockIdx.x) * 4 + wave;
  if (t >= T) return;
  float v[V], p[V], b[V] = {};
  load_logits<V>(logits + (long)t * a.E, a.E, lane, v);
  if (bias) load_row<V>(bias, a.E, lane, 0.f, b);
  double e[V];
  if (a.sigmoid) {
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = (double)fmaxf(-fabsf(v[j]), -110.f);  // (e^-110 is 0 in float32)
    exp_below<V>(e);
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = (float)((v[j] < 0.f ? e[j] : 1.0) * reciprocal(1.0 + e[j]));
  } else {
    int m = key_of(v[0]);
#pragma unroll
    for (int j = 1; j < V; ++j) m = max(m, key_of(v[j]));
    // (a row that is all masked: nothing is selected, whatever the scores are)
    const float top = fmaxf(of_key(wave_max_int(m)), -3.4028234664e38f);
    // (e^-110 is 0 in float32, and what masked experts add to a sum of at least 1 stays below 64 bits)
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = fmax((double)v[j] - (double)top, -110.0);
    exp_below<V>(e);
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) sum += e[j];
    const double inv = reciprocal(fmax(wave_sum_double(sum), 1.0));
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = (float)(e[j] * inv);
  }
  int c[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float x = p[j] + fmaxf(b[j], -INFINITY);  // (a bias of NaN as -infinity)
    c[j] = v[j] == -INFINITY ? kNone : key_of(x);
  }
  if (a.kept < a.groups) {
    int* s = lds[wave];
#pragma unroll
    for (int j = 0; j < V; ++j) s[lane + 64 * j] = c[j];
    // (one wavefront's own LDS words: written and read in program order)
    __builtin_amdgcn_wave_barrier();
    // 2^log lanes a group find its two largest
    const int per = a.E / a.groups, log = 31 - __clz(64 / a.groups), L = 1 << log;
    const int g = lane >> log, sub = lane & (L - 1);
    int first = kNone, second = kNone;
    if (g < a.groups) {
      for (int i = sub; i < per; i += L) {
        const int x = s[g * per + i];
        second = max(second, min(first, x));
        first = max(first, x);
      }
    }
    auto join = [&](uint32_t f, uint32_t q) {
      second = max(max(second, (int)q), min(first, (int)f));
      first = max(first, (int)f);
    };
    if (log > 0) join(dpp_from<kDppXor1>(first), dpp_from<kDppXor1>(second));
    if (log > 1) join(dpp_from<kDppXor2>(first), dpp_from<kDppXor2>(second));
    if (log > 2) join(dpp_from<kDppHalf>(first), dpp_from<kDppHalf>(second));
    if (log > 3) join(dpp_from<kDppRow>(first), dpp_from<kDppRow>(second));
    if (log > 4) join(__shfl_xor(first, 16), __shfl_xor(second, 16));
    const int score = a.group_top == 2 && second > kNone ? key_of(of_key(first) + of_key(second)) : first;
    // a group stays if fewer than `kept` are larger, or equal and in front of it: a group's lanes share the others
    __builtin_amdgcn_wave_barrier();
    if (sub == 0 && g < a.groups) s[g] = score;
    __builtin_amdgcn_wave_barrier();
    int before = 0;
    for (int q = sub; q < a.groups; q += L) before += s[q] > score - (q < g);
    if (log > 0) before += dpp_from<kDppXor1>(before);
    if (log > 1) before += dpp_from<kDppXor2>(before);
    if (log > 2) before += dpp_from<kDppHalf>(before);
    if (log > 3) before += dpp_from<kDppRow>(before);
    if (log > 4) before += __shfl_xor(before, 16);
    const unsigned long long stays = __ballot(before < a.kept);
    // (e / per by a product: exact for e < 1024 and per <= 1024)
    const uint32_t by = (1u << 20) / (uint32_t)per + 1u;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int x = lane + 64 * j;
      if (x < a.E && !(stays >> (((x * by) >> 20) << log) & 1ull)) c[j] = kNone;
    }
    __builtin_amdgcn_wave_barrier();
  }
#pragma unroll
  for (int j = 0; j < V; ++j) lds[wave][lane + 64 * j] = __float_as_int(p[j]);
  constexpr int KV = MANY ? V : 1;
  int pe[KV];
#pragma unroll
  for (int j = 0; j < KV; ++j) pe[j] = -1;
  auto largest = [&]() {
    int m = c[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = max(m, c[j]);
    return __builtin_amdgcn_readfirstlane(wave_max_int(m));
  };
  int m = largest();
  for (int r = 0; r < a.k && m != kNone; ++r) {  // (kNone: only masked experts are left)
    bool found = false;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const unsigned long long at = __ballot(c[j] == m);
      if (!found && at) {
        const int l = __ffsll((long long)at) - 1;
        c[j] = lane == l ? kNone : c[j];
        found = true;
#pragma unroll
        for (int i = 0; i < KV; ++i)
          if (i == r >> 6) pe[i] = lane == (r & 63) ? l + 64 * j : pe[i];
      }
    }
    m = largest();
  }
  __builtin_amdgcn_wave_barrier();
  float x[KV], sum = 0.f;
#pragma unroll
  for (int j = 0; j < KV; ++j) {
    x[j] = pe[j] < 0 ? 0.f : __int_as_float(lds[wave][pe[j]]);
    sum += x[j];
  }
  if (a.normalize) {
    sum = wave_sum_float(sum);
#pragma unroll
    for (int j = 0; j < KV; ++j) x[j] = sum > 0.f ? x[j] / sum : 0.f;
  }
#pragma unroll
  for (int j = 0; j < KV; ++j) {
    const int r = lane + 64 * j;
    if (r < a.k) {
      idx[(long)t * a.k + r] = pe[j];
      w[(long)t * a.k + r] = x[j] * a.scale;
    }
  }
}

// One wavefront per token.  With s the scores, u = s at the slots (0 for masked
// or outside ones), S = sum u, g the slots' gradients and D_e the sum over the
// slots of e:
//   as they are:    sigmoid   gl_e = scale D_e s_e (1 - s_e)      softmax   gl_e = scale s_e (D_e - sum_i u_i g_i)
//   renormalised:   with g_i - sum_j u_j g_j / S in the place of g_i and s_e / S in the place of the first s_e, where the
//                   softmax's sum is 0 by itself (all 0 where S is)
// The differences cancel: renormalised, one slot has a gradient of 0, and where one
// holds nearly all of S (or of the softmax) what is left is far below the g's.  So
// scores, sums and differences are float64, and a result is rounded once, at its
// end.  (A score that is 0 in float32, as the forward pass has it, is 0.)
// A lane adds up its experts' slots in slot order (no atomics; the same expert
// twice counts twice); a slot's score comes from the lane that holds it.  8192 x
// 128, 8 slots: 7.4 us (sigmoid), 7.9 (softmax); 16384 x 256, 6 slots, softmax:
// 17.2 us, where its bytes take 6.7 (in float32 6.9, 7.0 and 13.9).
template <int V>
__global__ void __launch_bounds__(256) qmoe_route_scored_grad(const float* __restrict__ gw,
                                                              const float* __restrict__ logits,
                                                              const void* __restrict__ idx, bool idx64, int T,
                                                              RouteScored a, int b0, float* __restrict__ gl) {
  extern __shared__ double smem[];  // per wavefront: k values; behind all of those, per wavefront: k experts
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  double* sv = smem + wave * a.k;
  int* se = reinterpret_cast<int*>(smem + 4 * a.k) + wave * a.k;
  const int t = (b0 + blockIdx.x) * 4 + wave;
  if (t >= T) return;
  float v[V];
  load_logits<V>(logits + (long)t * a.E, a.E, lane, v);
  // p: scores (masked: -1); c: 1 - p of the sigmoid (from e^-|l|, which keeps its digits), 1 of the softmax
  double p[V], c[V];
  auto held = [](double s) { return (float)s > 0.f ? s : 0.0; };
  if (a.sigmoid) {
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = (double)fmaxf(-fabsf(v[j]), -110.f);
    exp_below<V>(p);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const double near1 = reciprocal(1.0 + p[j]), near0 = held(p[j] * near1);
      p[j] = v[j] < 0.f ? near0 : near1;
      c[j] = v[j] < 0.f ? near1 : near0;
    }
  } else {
    int m = key_of(v[0]);
#pragma unroll
    for (int j = 1; j < V; ++j) m = max(m, key_of(v[j]));
    const float top = fmaxf(of_key(wave_max_int(m)), -3.4028234664e38f);
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = fmax((double)v[j] - (double)top, -110.0);
    exp_below<V>(p);
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) sum += p[j];
    const double inv = reciprocal(fmax(wave_sum_double(sum), 1.0));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      p[j] = held(p[j] * inv);
      c[j] = 1.0;
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) p[j] = v[j] == -INFINITY ? -1.0 : p[j];
  // (renormalised: the slots' gradients from the first held one's, so that a single slot leaves exactly 0)
  double S = 0.0, dot = 0.0, g0 = 0.0;
  bool first = a.normalize;
  for (int s0 = 0; s0 < a.k; s0 += 64) {  // (every lane stays: its scores are read)
    const int s = s0 + lane;
    const long at = (long)t * a.k + min(s, a.k - 1);
    const int64_t i64 = idx64 ? static_cast<const int64_t*>(idx)[at] : static_cast<const int*>(idx)[at];
    const float g = gw[at];
    const int i = i64 >= 0 && i64 < a.E ? (int)i64 : -1;
    double u = -1.0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const double x = __shfl(p[j], i & 63);
      u = i >> 6 == j ? x : u;
    }
    const bool on = s < a.k && u >= 0.0;
    const unsigned long long all = __ballot(on);
    if (first && all) {
      g0 = (double)__shfl(g, __ffsll((long long)all) - 1);
      first = false;
    }
    if (s >= a.k) continue;
    u = on ? u : 0.0;
    const double x = on ? (double)g - g0 : 0.0;
    se[s] = on ? i : -1;
    sv[s] = x;
    S += u;
    dot = fma(u, x, dot);
  }
  S = wave_sum_double(S);
  dot = wave_sum_double(dot);
  double shift = 0.0, mean = dot, over = 1.0;
  if (a.normalize) {
    over = S > 0.0 ? reciprocal(S) : 0.0;
    shift = dot * over;
    mean = 0.0;
  }
  // (one wavefront's own LDS words: written and read in program order)
  __builtin_amdgcn_wave_barrier();
  double d[V];
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = 0.0;
  for (int s = 0; s < a.k; ++s) {
    const int i = se[s];
    const double x = sv[s] - shift;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (i == lane + 64 * j) d[j] += x;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (lane + 64 * j >= a.E) continue;
    const double o = p[j] < 0.0 ? 0.0 : p[j] * over * c[j] * (d[j] - (a.sigmoid ? 0.0 : mean)) * (double)a.scale;
    gl[(long)t * a.E + lane + 64 * j] = (float)o;
  }
}

template <int V>
void go_scored(dim3 grid, hipStream_t st, const float* logits, const float* bias, int T, const RouteScored& a, int b0,
               int* idx, float* w) {
  if (a.k <= 64)
    hipLaunchKernelGGL((qmoe_route_scored<V, false>), grid, dim3(256), 0, st, logits, bias, T, a, b0, idx, w);
  else
    hipLaunchKernelGGL((qmoe_route_scored<V, true>), grid, dim3(256), 0, st, logits, bias, T, a, b0, idx, w);
}

}  // namespace

#define QMOE_BY_REGS(CALL)                                  \
  {                                                         \
    const int v_ = (a.E + 63) / 64;                         \
    if (v_ <= 1) CALL(1);                                   \
    else if (v_ <= 2) CALL(2);                              \
    else if (v_ <= 4) CALL(4);                              \
    else if (v_ <= 8) CALL(8);                              \
    else CALL(16);                                          \
  }

hipError_t launch_route_scored(const float* logits, const float* bias, int T, const RouteScored& a, int* idx, float* w,
                               hipStream_t st) {
  return in_launches(((long)T + 3) / 4, [&](int b0, unsigned n) {
    const dim3 grid(n);
#define QMOE_CALL(VV) go_scored<VV>(grid, st, logits, bias, T, a, b0, idx, w)
    QMOE_BY_REGS(QMOE_CALL)
#undef QMOE_CALL
  });
}

hipError_t launch_route_scored_grad(const float* gw, const float* logits, const void* idx, bool idx64, int T,
                                    const RouteScored& a, float* gl, hipStream_t st) {
  const size_t lds = (size_t)4 * a.k * (sizeof(double) + sizeof(int));
  return in_launches(((long)T + 3) / 4, [&](int b0, unsigned n) {
    const dim3 grid(n), block(256);
#define QMOE_CALL(VV) \
  hipLaunchKernelGGL(qmoe_route_scored_grad<VV>, grid, block, lds, st, gw, logits, idx, idx64, T, a, b0, gl)
    QMOE_BY_REGS(QMOE_CALL)
#undef QMOE_CALL
  });
}

}  // namespace qmoe
