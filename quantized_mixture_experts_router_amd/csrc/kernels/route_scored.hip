// Routing from scores (route_scored.h).
#include <math.h>

#include "common.hpp"
#include "launches.h"
#include "route_scored.h"

namespace qmoe {

namespace {

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// A row's logits, lane + 64 j: +infinity counts as the largest float, -infinity
// and NaN (masked) come back as -infinity.
template <int V>
__device__ __forceinline__ void load_logits(const float* __restrict__ row, int E, int lane, float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float x = lane + 64 * j < E ? row[lane + 64 * j] : -INFINITY;
    v[j] = x != x ? -INFINITY : fminf(x, 3.4028234664e38f);
  }
}

// One wavefront per token, expert lane + 64 j in register j.  The scores are
// evaluated in 64 bits and rounded once to float32: an expert is selected by
// comparing its score plus bias with others', and two that differ in float32's
// last bits would change places with the rounding errors of a float32 exponential.
template <int V>
__global__ void __launch_bounds__(256) qmoe_route_scored(const float* __restrict__ logits,
                                                         const float* __restrict__ bias, int T, RouteScored a, int b0,
                                                         int* __restrict__ idx, float* __restrict__ w) {
  __shared__ float sc[4][64 * V];
  const int wave = threadIdx.x >> 6, lane = lane_id();
  const int t = (b0 + blockIdx.x) * 4 + wave;
  if (t >= T) return;
  float v[V], p[V], c[V];
  load_logits<V>(logits + (long)t * a.E, a.E, lane, v);
  if (a.sigmoid) {
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = (float)(1.0 / (1.0 + exp(-(double)v[j])));
  } else {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, v[j]);
    m = wave_max(m);
    if (m == -INFINITY) m = 0.f;
    double e[V], sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      e[j] = exp((double)v[j] - (double)m);
      sum += e[j];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = (float)(e[j] / sum);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    c[j] = p[j];
    if (bias && lane + 64 * j < a.E) c[j] += bias[lane + 64 * j];
    c[j] = v[j] == -INFINITY || c[j] != c[j] ? -INFINITY : c[j];
  }
  if (a.kept < a.groups) {
    float* s = sc[wave];
#pragma unroll
    for (int j = 0; j < V; ++j) s[lane + 64 * j] = c[j];
    // (one wavefront's own LDS words: written and read in program order)
    __builtin_amdgcn_wave_barrier();
    // 2^log lanes a group find its two largest
    const int per = a.E / a.groups, log = 31 - __clz(64 / a.groups), L = 1 << log;
    const int g = lane >> log;
    float first = -INFINITY, second = -INFINITY;
    if (g < a.groups) {
      for (int i = lane & (L - 1); i < per; i += L) {
        const float x = s[g * per + i];
        second = fmaxf(second, fminf(first, x));
        first = fmaxf(first, x);
      }
    }
    for (int o = 1; o < L; o <<= 1) {
      const float f = __shfl_xor(first, o), q = __shfl_xor(second, o);
      second = fmaxf(fmaxf(second, q), fminf(first, f));
      first = fmaxf(first, f);
    }
    const float score = a.group_top == 2 && second > -INFINITY ? first + second : first;
    // a group stays if fewer than `kept` are larger, or equal and in front of it
    int before = 0;
    for (int q = 0; q < a.groups; ++q) {
      const float o = __shfl(score, q << log);
      before += o > score || (o == score && q < g);
    }
    const unsigned long long stays = __ballot(before < a.kept);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = lane + 64 * j;
      if (e < a.E && !(stays >> ((e / per) << log) & 1ull)) c[j] = -INFINITY;
    }
  }
  // pick r waits in lane r % 64 of register r / 64
  float pv[V], sum = 0.f;
  int pe[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    pv[j] = 0.f;
    pe[j] = -1;
  }
  for (int r = 0; r < a.k; ++r) {
    float m = c[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, c[j]);
    m = wave_max(m);
    if (m == -INFINITY) break;  // only masked experts are left
    int e = -1;
    float at = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const unsigned long long b = __ballot(c[j] == m);
      if (e < 0 && b) {
        const int l = __ffsll((long long)b) - 1;
        e = l + 64 * j;
        at = __shfl(p[j], l);
        if (lane == l) c[j] = -INFINITY;
      }
    }
    sum += at;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (r == lane + 64 * j) {
        pv[j] = at;
        pe[j] = e;
      }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int r = lane + 64 * j;
    if (r < a.k) {
      float x = pv[j];
      if (a.normalize) x = sum > 0.f ? x / sum : 0.f;
      idx[(long)t * a.k + r] = pe[j];
      w[(long)t * a.k + r] = x * a.scale;
    }
  }
}

// One wavefront per token.  With s the scores, u = s at the slots (0 for masked
// or outside ones), S = sum u, g the slots' gradients times scale and D_e the sum
// over the slots of e:
//   as they are:    sigmoid   gl_e = D_e s_e (1 - s_e)      softmax   gl_e = s_e (D_e - sum_i u_i g_i)
//   renormalised:   with g_i - sum_i u_i g_i / S in the place of g_i and s_e / S in the place of the first s_e, where the
//                   softmax's sum is 0 by itself (all 0 where S is)
// A lane adds up its experts' slots in slot order (no atomics; the same expert
// twice counts twice).
template <int V>
__global__ void __launch_bounds__(256) qmoe_route_scored_grad(const float* __restrict__ gw,
                                                              const float* __restrict__ logits,
                                                              const void* __restrict__ idx, bool idx64, int T,
                                                              RouteScored a, int b0, float* __restrict__ gl) {
  extern __shared__ char smem[];  // per wavefront: k experts, k values
  const int wave = threadIdx.x >> 6, lane = lane_id();
  int* se = reinterpret_cast<int*>(smem) + wave * 2 * a.k;
  float* sv = reinterpret_cast<float*>(se + a.k);
  const int t = (b0 + blockIdx.x) * 4 + wave;
  if (t >= T) return;
  const float* row = logits + (long)t * a.E;
  float v[V];
  load_logits<V>(row, a.E, lane, v);
  float top = 0.f, inv = 1.f;
  if (!a.sigmoid) {
    float m = v[0], sum = 0.f;
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, v[j]);
    m = wave_max(m);
    top = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < V; ++j) sum += expf(v[j] - top);
    sum = wave_sum(sum);
    inv = sum > 0.f ? 1.f / sum : 0.f;
  }
  // (sigmoid: e^-|l| keeps the digits of scores near 0 and of 1 - s near 1)
  auto score = [&](float l) {
    if (!a.sigmoid) return expf(l - top) * inv;
    const float e = expf(-fabsf(l));
    return (l < 0.f ? e : 1.f) / (1.f + e);
  };
  float S = 0.f, dot = 0.f;
  for (int s = lane; s < a.k; s += 64) {
    const long at = (long)t * a.k + s;
    int64_t e = idx64 ? static_cast<const int64_t*>(idx)[at] : static_cast<const int*>(idx)[at];
    float x = -INFINITY;
    if (e >= 0 && e < a.E) {
      x = row[e];
      x = x != x ? -INFINITY : fminf(x, 3.4028234664e38f);
    }
    if (x == -INFINITY) e = -1;
    const float u = e < 0 ? 0.f : score(x), g = e < 0 ? 0.f : gw[at] * a.scale;
    se[s] = (int)e;
    sv[s] = g;
    S += u;
    dot = fmaf(u, g, dot);
  }
  S = wave_sum(S);
  dot = wave_sum(dot);
  float shift = 0.f, mean = dot;
  if (a.normalize) {
    shift = S > 0.f ? dot / S : 0.f;
    mean = 0.f;
  }
  // (one wavefront's own LDS words: written and read in program order)
  __builtin_amdgcn_wave_barrier();
  float d[V];
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = 0.f;
  for (int s = 0; s < a.k; ++s) {
    const int e = se[s];
    const float x = sv[s] - shift;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (e == lane + 64 * j) d[j] += x;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (lane + 64 * j >= a.E) continue;
    float o = 0.f;
    if (v[j] != -INFINITY) {
      float f = score(v[j]);
      // (an expert that no slot names may be far above the selection's sum: s / S would pass float32)
      if (a.normalize) f = S > 0.f && d[j] != 0.f ? f / S : 0.f;
      if (a.sigmoid) f *= score(-v[j]);
      o = f * (d[j] - (a.sigmoid ? 0.f : mean));
    }
    gl[(long)t * a.E + lane + 64 * j] = o;
  }
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
    const dim3 grid(n), block(256);
#define QMOE_CALL(VV) hipLaunchKernelGGL(qmoe_route_scored<VV>, grid, block, 0, st, logits, bias, T, a, b0, idx, w)
    QMOE_BY_REGS(QMOE_CALL)
#undef QMOE_CALL
  });
}

hipError_t launch_route_scored_grad(const float* gw, const float* logits, const void* idx, bool idx64, int T,
                                    const RouteScored& a, float* gl, hipStream_t st) {
  const size_t lds = (size_t)4 * 2 * a.k * 4;
  return in_launches(((long)T + 3) / 4, [&](int b0, unsigned n) {
    const dim3 grid(n), block(256);
#define QMOE_CALL(VV) \
  hipLaunchKernelGGL(qmoe_route_scored_grad<VV>, grid, block, lds, st, gw, logits, idx, idx64, T, a, b0, gl)
    QMOE_BY_REGS(QMOE_CALL)
#undef QMOE_CALL
  });
}

}  // namespace qmoe
