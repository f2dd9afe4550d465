// C ABI of the linear layers (declared in include/qmoe.h): contract check,
// workspace plan and enqueue, forward and backward.
//
// Forward:  [row padding] -> matrix kernel (epilogue inside, or fp32 sums per
//           range of K -> finishing pass)
// Backward: [row padding] -> activation gradient with column sums -> bias
//           gradient -> grad_input product -> grad_weights product
// with every intermediate in the caller's workspace.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>

#include "kernels/linear.h"
#include "qmoe.h"

using namespace qmoe;

namespace {

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int64_t kMaxGroups = 1023;
constexpr int64_t kMaxRow = int64_t(1) << 20;   // K and N: a tile's rows stay inside one 32-bit buffer range
constexpr int64_t kMaxRows = int64_t(1) << 30;  // M

struct LinPlan {
  int64_t M = 0, K = 0, N = 0, No = 0, G = 1;
  bool grouped = false;
  int type = LIN_F32;
  int64_t es = 4, Kp = 0, Np = 0;  // element size; K and N in whole 16-byte runs
  LinearAct act{};
  LinearPlan fwd{LT_32x128, 1}, dx{LT_32x128, 1}, dw{LT_32x128, 1};
  size_t off_x = 0, off_w = 0, off_dz = 0, off_sums = 0, off_partial = 0;
  size_t bytes = 0;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tile shape and ranges of the reduction for a product of `rows` output rows
// (of `groups` groups, the rows spread over them evenly as far as the host
// can know) by `cols` columns summed over `red`: the least of an estimate in
// microseconds.  A compute unit runs ceil(items / 256) items one after the
// other; an item costs its stages (128 bytes of r a row) and a fixed part
// (first loads, output).  Both were measured on full cards: 4096 x 4096
// outputs, K = 4096, at 1.25 PFLOP/s (256 x 256), 0.91 (128 x 128), 0.81
// (64 x 128) and 0.58 (32 x 128) in bfloat16, 139, 141 and 135 TFLOP/s in
// float32.  Ranges add the float32 sums' way to memory and back and one more
// launch.
// Against every tile in 1 to 32 ranges, each timed (755 sizes: 1 to 8192 rows,
// reductions and columns 256 to 16384, dense and 4 to 64 groups): the choice is
// 0.4 to 2.6 % above the best at the median, by product and type, and within
// 15 to 26 % in nine of ten.  It is furthest off where many groups share a few
// rows (1 row in 64 groups, 60 against 21 us: too many ranges) and where the
// products of a few hundred rows would rather take large tiles in ranges (326 x
// 11912 -> 1320, 68 against 33 us).
LinearPlan plan_product(int type, int64_t rows, int64_t groups, int64_t cols, int64_t red) {
  static const struct {
    int tile;
    int64_t bq, bp;
    double stage16, stage32, fixed;
  } tiles[] = {{LT_256x256, 256, 256, 1.60, 0.0, 6.0},
               {LT_128x128, 128, 128, 0.60, 1.93, 2.5},
               {LT_64x128, 64, 128, 0.33, 0.95, 1.4},
               {LT_32x128, 32, 128, 0.23, 0.50, 0.9}};
  const int64_t cus = 256, bk = type == LIN_F32 ? 32 : 64;
  const int64_t per = std::max<int64_t>(1, ceil_div(rows, groups)), stages = std::max<int64_t>(1, ceil_div(red, bk));
  LinearPlan best{LT_32x128, 1};
  double best_cost = -1;
  for (const auto& t : tiles) {
    const double stage = type == LIN_F32 ? t.stage32 : t.stage16;
    if (stage == 0.0) continue;
    const int64_t n = ceil_div(per, t.bq) * std::min(groups, rows) * ceil_div(cols, t.bp);
    for (int64_t s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
      if (s > 1 && stages < 4 * s) break;  // at least four stages a range
      if (s > 1 && rows * (cols + 3) >= int64_t(1) << 31) break;  // (the finishing pass counts outputs in 32 bits)
      // (alone on its compute unit a float32 item leaves the matrix cores a fifth idle; without this factor the products
      // whose plan it changes take 9 % longer, geometric mean over 8717, 6 % at the median)
      const double slow = type == LIN_F32 && n * s <= cus ? 1.2 : 1.0;
      double cost = (double)ceil_div(n * s, cus) * (t.fixed + (double)ceil_div(stages, s) * stage * slow);
      if (s > 1) cost += 4.0 + (double)s * (double)rows * (double)cols * 8.0 / 4.5e6;
      if (best_cost < 0 || cost < best_cost) {
        best_cost = cost;
        best.tile = t.tile;
        best.splits = (int)s;
      }
    }
  }
  return best;
}

int64_t numel(const qmoe_tensor* t) {
  int64_t n = 1;
  for (int i = 0; i < t->rank; ++i) n *= t->dims[i];
  return n;
}

qmoe_status check_act(const qmoe_linear_attrs* a, LinearAct* act) {
  if (a->activation_type < QMOE_ACT_RELU || a->activation_type > QMOE_ACT_IDENTITY) return QMOE_ERR_ATTR;
  if (a->swiglu_fusion < 0 || a->swiglu_fusion > 2) return QMOE_ERR_ATTR;
  if (a->activation_type == QMOE_ACT_SWIGLU) {
    if (a->swiglu_fusion != 1) return QMOE_ERR_UNSUPPORTED;
    if (a->has_swiglu_limit != 0 && a->has_swiglu_limit != 1) return QMOE_ERR_ATTR;
    if (a->has_swiglu_limit && !(a->swiglu_limit > 0.f)) return QMOE_ERR_ATTR;
  }
  act->type = a->activation_type;
  act->alpha = a->activation_alpha;
  act->beta = a->activation_beta;
  act->has_limit = a->has_swiglu_limit;
  act->limit = a->swiglu_limit;
  return QMOE_OK;
}

// The shapes shared by both directions: rows [M, K] (input), weights, an
// output-shaped tensor [M, No], and the optional ones.
qmoe_status check(const qmoe_tensor* input, const qmoe_tensor* weights, const qmoe_tensor* bias,
                  const qmoe_tensor* offsets, const qmoe_tensor* preact, const qmoe_linear_attrs* attrs,
                  std::initializer_list<const qmoe_tensor*> out_like, LinPlan* p) {
  if (!input || !weights || !attrs) return QMOE_ERR_NULL;
  if (input->rank != 2 || (weights->rank != 2 && weights->rank != 3)) return QMOE_ERR_SHAPE;
  p->grouped = weights->rank == 3;
  if (p->grouped && !offsets) return QMOE_ERR_NULL;
  if (!p->grouped && offsets) return QMOE_ERR_SHAPE;
  if (bias && bias->rank != (p->grouped ? 2 : 1)) return QMOE_ERR_SHAPE;
  if (offsets && offsets->rank != 1) return QMOE_ERR_SHAPE;
  if (preact && preact->rank != 2) return QMOE_ERR_SHAPE;
  for (const qmoe_tensor* t : out_like)
    if (t && t->rank != 2) return QMOE_ERR_SHAPE;
  const int32_t T = input->dtype;
  if (T != QMOE_F32 && T != QMOE_F16 && T != QMOE_BF16) return QMOE_ERR_DTYPE;
  if (weights->dtype != T || (bias && bias->dtype != T) || (preact && preact->dtype != T)) return QMOE_ERR_DTYPE;
  for (const qmoe_tensor* t : out_like)
    if (t && t->dtype != T) return QMOE_ERR_DTYPE;
  if (offsets && offsets->dtype != QMOE_I32) return QMOE_ERR_DTYPE;
  const qmoe_tensor* ts[] = {input, weights, bias, offsets, preact};
  for (const qmoe_tensor* t : ts)
    if (t)
      for (int i = 0; i < t->rank; ++i)
        if (t->dims[i] < 0) return QMOE_ERR_SHAPE;
  const qmoe_status st = check_act(attrs, &p->act);
  if (st != QMOE_OK) return st;
  const int d = p->grouped ? 1 : 0;
  p->M = input->dims[0];
  p->K = input->dims[1];
  p->G = p->grouped ? weights->dims[0] : 1;
  p->N = weights->dims[d];
  if (weights->dims[d + 1] != p->K) return QMOE_ERR_SHAPE;
  if (offsets && offsets->dims[0] != p->G + 1) return QMOE_ERR_SHAPE;
  if (bias && (bias->dims[d] != p->N || (p->grouped && bias->dims[0] != p->G))) return QMOE_ERR_SHAPE;
  if (preact && (preact->dims[0] != p->M || preact->dims[1] != p->N)) return QMOE_ERR_SHAPE;
  p->No = p->N;
  if (p->act.type == QMOE_ACT_SWIGLU) {
    if (p->N % 2 != 0) return QMOE_ERR_SHAPE;
    p->No = p->N / 2;
  }
  for (const qmoe_tensor* t : out_like)
    if (t && (t->dims[0] != p->M || t->dims[1] != p->No)) return QMOE_ERR_SHAPE;
  if (p->G > kMaxGroups || p->M > kMaxRows || p->K > kMaxRow || p->N > kMaxRow) return QMOE_ERR_UNSUPPORTED;
  // one workgroup per tile and column block, tiles as small as 32 rows by 128
  // columns, the passes one per 256 columns of 64 rows: their indices (and
  // nine q blocks more) stay within 32 bits
  const int64_t wide = std::max(p->N, p->K);
  if ((p->M / 32 + 9 + p->G) * (wide / 128 + 1) >= (int64_t(1) << 31) - 512 ||
      ((p->N / 32 + 1) * p->G + 8) * (p->K / 128 + 1) >= (int64_t(1) << 31) - 512)
    return QMOE_ERR_UNSUPPORTED;
  p->type = T == QMOE_F32 ? LIN_F32 : T == QMOE_F16 ? LIN_F16 : LIN_BF16;
  p->es = T == QMOE_F32 ? 4 : 2;
  const int64_t run = 16 / p->es;
  p->Kp = ceil_div(p->K, run) * run;
  p->Np = ceil_div(p->N, run) * run;
  return QMOE_OK;
}

int64_t wrows(const LinPlan& p) { return p.G * p.N; }

void place_forward(LinPlan* p) {
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align256(o + bytes); return at; };
  if (p->M == 0 || p->N == 0) return;
  if (p->Kp != p->K) {
    p->off_x = take((size_t)(p->M * p->Kp * p->es));
    p->off_w = take((size_t)(wrows(*p) * p->Kp * p->es));
  }
  p->fwd = plan_product(p->type, p->M, std::max<int64_t>(1, p->G), p->N, p->K);
  if (p->fwd.splits > 1) p->off_partial = take(sizeof(float) * (size_t)(p->fwd.splits * p->M * ceil_div(p->N, 4) * 4));
  p->bytes = o;
}

bool needs_dz(const LinPlan& p) { return p.act.type != QMOE_ACT_IDENTITY || p.Np != p.N; }

void place_backward(LinPlan* p, bool gx, bool gw, bool gb) {
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align256(o + bytes); return at; };
  if (p->Kp != p->K) {
    if (gw) p->off_x = take((size_t)(p->M * p->Kp * p->es));
    if (gx) p->off_w = take((size_t)(wrows(*p) * p->Kp * p->es));
  }
  if ((gx || gw) && needs_dz(*p)) p->off_dz = take((size_t)(p->M * p->Np * p->es));
  if (gb) p->off_sums = take(sizeof(float) * (size_t)(linear_sum_blocks(p->M, p->grouped ? p->G : -1) * p->N));
  size_t part = 0;
  const int64_t Kq = ceil_div(p->K, 4) * 4;
  if (gx) {
    p->dx = plan_product(p->type, std::max<int64_t>(1, p->M), std::max<int64_t>(1, p->G), p->K, p->N);
    if (p->dx.splits > 1) part = sizeof(float) * (size_t)(p->dx.splits * p->M * Kq);
  }
  if (gw) {
    p->dw = plan_product(p->type, std::max<int64_t>(1, wrows(*p)), std::max<int64_t>(1, p->G), p->K,
                         ceil_div(p->M, std::max<int64_t>(1, p->G)));
    if (p->dw.splits > 1) part = std::max(part, sizeof(float) * (size_t)(p->dw.splits * wrows(*p) * Kq));
  }
  if (part) p->off_partial = take(part);
  p->bytes = o;
}

qmoe_status check_grads(const qmoe_tensor* grad_output, const qmoe_tensor* input, const qmoe_tensor* weights,
                        const qmoe_tensor* preact, const qmoe_tensor* offsets, const qmoe_linear_attrs* attrs,
                        const qmoe_tensor* grad_input, const qmoe_tensor* grad_weights, const qmoe_tensor* grad_bias,
                        LinPlan* p) {
  if (!grad_output) return QMOE_ERR_NULL;
  const qmoe_status st = check(input, weights, grad_bias, offsets, preact, attrs, {grad_output}, p);
  if (st != QMOE_OK) return st;
  if (p->act.type != QMOE_ACT_IDENTITY && !preact) return QMOE_ERR_NULL;
  if (grad_input) {
    if (grad_input->dtype != input->dtype) return QMOE_ERR_DTYPE;
    if (grad_input->rank != 2 || grad_input->dims[0] != p->M || grad_input->dims[1] != p->K) return QMOE_ERR_SHAPE;
  }
  if (grad_weights) {
    if (grad_weights->dtype != input->dtype) return QMOE_ERR_DTYPE;
    if (grad_weights->rank != weights->rank) return QMOE_ERR_SHAPE;
    for (int i = 0; i < weights->rank; ++i)
      if (grad_weights->dims[i] != weights->dims[i]) return QMOE_ERR_SHAPE;
  }
  place_backward(p, grad_input != nullptr, grad_weights != nullptr, grad_bias != nullptr);
  return QMOE_OK;
}

// Pointers present where there are elements, and aligned: operands of the
// matrix kernel to 16 bytes when their rows are whole 16-byte runs (they are
// copied to such rows otherwise), everything else to the element.
qmoe_status check_data(std::initializer_list<const qmoe_tensor*> ts, int64_t es) {
  for (const qmoe_tensor* t : ts) {
    if (!t) continue;
    if (numel(t) > 0 && !t->data) return QMOE_ERR_NULL;
    if (!aligned_to(t->data, (uintptr_t)es)) return QMOE_ERR_ALIGN;
  }
  return QMOE_OK;
}

qmoe_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return QMOE_OK;
  if (!ws) return QMOE_ERR_NULL;
  if (have < need) return QMOE_ERR_WORKSPACE;
  return aligned_to(ws, 256) ? QMOE_OK : QMOE_ERR_ALIGN;
}

// One product: matrix kernel, and the finishing pass when it ran in ranges.
bool run_product(int type, int mode, const LinearPlan& pl, LinearGemm g, float* partial, hipStream_t s) {
  g.splits = pl.splits;
  g.partial = partial;
  if (launch_linear(type, mode, pl.tile, g, s) != hipSuccess) return false;
  return pl.splits == 1 || launch_linear_finish(type, mode, g, s) == hipSuccess;
}

LinearGemm base_gemm(const LinPlan& p, const qmoe_tensor* input, const qmoe_tensor* weights,
                     const qmoe_tensor* offsets) {
  LinearGemm g{};
  g.x = input->data;
  g.w = weights->data;
  g.ldx = g.ldw = p.K;
  g.lddz = p.N;
  g.offsets = offsets ? static_cast<const int*>(offsets->data) : nullptr;
  g.G = (int)p.G;
  g.M = (int)p.M;
  g.N = (int)p.N;
  g.K = (int)p.K;
  g.act = p.act;
  return g;
}

}  // namespace

extern "C" {

void qmoe_linear_attrs_default(qmoe_linear_attrs* a) {
  a->activation_type = QMOE_ACT_IDENTITY;
  a->swiglu_fusion = 0;
  a->activation_alpha = 1.f;
  a->activation_beta = 0.f;
  a->has_swiglu_limit = 0;
  a->swiglu_limit = 0.f;
}

qmoe_status qmoe_linear_plan_describe(const qmoe_tensor* input, const qmoe_tensor* weights, const qmoe_tensor* offsets,
                                      char* buf, size_t len) {
  if (!buf || len == 0) return QMOE_ERR_NULL;
  qmoe_linear_attrs a;
  qmoe_linear_attrs_default(&a);
  LinPlan p;
  const qmoe_status st = check(input, weights, nullptr, offsets, nullptr, &a, {}, &p);
  if (st != QMOE_OK) return st;
  place_forward(&p);
  place_backward(&p, true, true, true);
  auto tile = [](const LinearPlan& pl) {
    switch (pl.tile) {
      case LT_256x256: return "256x256";
      case LT_128x128: return "128x128";
      case LT_64x128: return "64x128";
    }
    return "32x128";
  };
  std::snprintf(buf, len, "forward=%s:%d grad_input=%s:%d grad_weights=%s:%d", tile(p.fwd), p.fwd.splits, tile(p.dx),
                p.dx.splits, tile(p.dw), p.dw.splits);
  return QMOE_OK;
}

qmoe_status qmoe_linear_workspace_size(const qmoe_tensor* input, const qmoe_tensor* weights, const qmoe_tensor* bias,
                                       const qmoe_tensor* residual, const qmoe_tensor* offsets,
                                       const qmoe_linear_attrs* attrs, const qmoe_tensor* output,
                                       const qmoe_tensor* preact, size_t* bytes) {
  if (!bytes) return QMOE_ERR_NULL;
  LinPlan p;
  const qmoe_status st = check(input, weights, bias, offsets, preact, attrs, {residual, output}, &p);
  if (st != QMOE_OK) return st;
  place_forward(&p);
  *bytes = p.bytes;
  return QMOE_OK;
}

qmoe_status qmoe_linear(const qmoe_tensor* input, const qmoe_tensor* weights, const qmoe_tensor* bias,
                        const qmoe_tensor* residual, const qmoe_tensor* offsets, const qmoe_linear_attrs* attrs,
                        const qmoe_tensor* output, const qmoe_tensor* preact, void* workspace, size_t workspace_bytes,
                        void* stream) {
  if (!output) return QMOE_ERR_NULL;
  LinPlan p;
  qmoe_status st = check(input, weights, bias, offsets, preact, attrs, {residual, output}, &p);
  if (st != QMOE_OK) return st;
  if (p.M == 0 || p.N == 0) return QMOE_OK;
  place_forward(&p);
  const uintptr_t op = p.Kp == p.K ? 16 : (uintptr_t)p.es;
  st = check_data({input, weights, bias, residual, output, preact}, p.es);
  if (st == QMOE_OK) st = check_data({offsets}, 4);
  if (st != QMOE_OK) return st;
  if (!aligned_to(input->data, op) || !aligned_to(weights->data, op)) return QMOE_ERR_ALIGN;
  st = check_ws(workspace, workspace_bytes, p.bytes);
  if (st != QMOE_OK) return st;

  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  LinearGemm g = base_gemm(p, input, weights, offsets);
  g.bias = bias ? bias->data : nullptr;
  g.res = residual ? residual->data : nullptr;
  g.out = const_cast<void*>(output->data);
  g.pre = preact ? const_cast<void*>(preact->data) : nullptr;
  if (p.Kp != p.K) {
    if (launch_linear_pad((int)p.es, {g.x, p.M, p.K, ws + p.off_x, p.Kp}, {g.w, wrows(p), p.K, ws + p.off_w, p.Kp}, s) !=
        hipSuccess)
      return QMOE_ERR_HIP;
    g.x = ws + p.off_x;
    g.w = ws + p.off_w;
    g.ldx = g.ldw = p.Kp;
  }
  return run_product(p.type, LIN_FWD, p.fwd, g, reinterpret_cast<float*>(ws + p.off_partial), s) ? QMOE_OK
                                                                                                : QMOE_ERR_HIP;
}

qmoe_status qmoe_linear_backward_workspace_size(const qmoe_tensor* grad_output, const qmoe_tensor* input,
                                                const qmoe_tensor* weights, const qmoe_tensor* preact,
                                                const qmoe_tensor* offsets, const qmoe_linear_attrs* attrs,
                                                const qmoe_tensor* grad_input, const qmoe_tensor* grad_weights,
                                                const qmoe_tensor* grad_bias, size_t* bytes) {
  if (!bytes) return QMOE_ERR_NULL;
  LinPlan p;
  const qmoe_status st = check_grads(grad_output, input, weights, preact, offsets, attrs, grad_input, grad_weights,
                                     grad_bias, &p);
  if (st != QMOE_OK) return st;
  *bytes = p.bytes;
  return QMOE_OK;
}

qmoe_status qmoe_linear_backward(const qmoe_tensor* grad_output, const qmoe_tensor* input, const qmoe_tensor* weights,
                                 const qmoe_tensor* preact, const qmoe_tensor* offsets,
                                 const qmoe_linear_attrs* attrs, const qmoe_tensor* grad_input,
                                 const qmoe_tensor* grad_weights, const qmoe_tensor* grad_bias, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  LinPlan p;
  qmoe_status st = check_grads(grad_output, input, weights, preact, offsets, attrs, grad_input, grad_weights,
                               grad_bias, &p);
  if (st != QMOE_OK) return st;
  st = check_data({grad_output, input, weights, preact, grad_input, grad_weights, grad_bias}, p.es);
  if (st == QMOE_OK) st = check_data({offsets}, 4);
  if (st != QMOE_OK) return st;
  const uintptr_t op = p.Kp == p.K ? 16 : (uintptr_t)p.es;
  if (!aligned_to(input->data, op) || !aligned_to(weights->data, op)) return QMOE_ERR_ALIGN;
  if (!needs_dz(p) && !aligned_to(grad_output->data, 16)) return QMOE_ERR_ALIGN;
  st = check_ws(workspace, workspace_bytes, p.bytes);
  if (st != QMOE_OK) return st;

  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool gx = grad_input && p.M > 0 && p.K > 0;
  const bool gw = grad_weights && p.G > 0 && p.N > 0 && p.K > 0;
  const bool gb = grad_bias && p.G > 0 && p.N > 0;
  LinearGemm g = base_gemm(p, input, weights, offsets);
  g.dz = grad_output->data;
  float* sums = gb ? reinterpret_cast<float*>(ws + p.off_sums) : nullptr;
  const bool dz = (gx || gw) && needs_dz(p);
  if (p.M > 0 && p.N > 0 && (dz || gb)) {
    LinearActGrad a{};
    a.dy = grad_output->data;
    a.z = p.act.type == QMOE_ACT_IDENTITY ? nullptr : preact->data;
    a.dz = dz ? ws + p.off_dz : nullptr;
    a.lddz = p.Np;
    a.sums = sums;
    a.offsets = g.offsets;
    a.G = g.G;
    a.M = g.M;
    a.N = g.N;
    a.act = p.act;
    if (launch_linear_act_grad(p.type, a, s) != hipSuccess) return QMOE_ERR_HIP;
    if (dz) {
      g.dz = ws + p.off_dz;
      g.lddz = p.Np;
    }
  }
  if (gb && launch_linear_bias_grad(p.type, sums, g.offsets, g.G, g.M, g.N, const_cast<void*>(grad_bias->data), s) !=
                hipSuccess)
    return QMOE_ERR_HIP;
  float* partial = reinterpret_cast<float*>(ws + p.off_partial);
  if (p.Kp != p.K) {
    if (launch_linear_pad((int)p.es, {g.x, gw ? p.M : 0, p.K, ws + p.off_x, p.Kp},
                          {g.w, gx ? wrows(p) : 0, p.K, ws + p.off_w, p.Kp}, s) != hipSuccess)
      return QMOE_ERR_HIP;
    g.x = ws + p.off_x;
    g.w = ws + p.off_w;
    g.ldx = g.ldw = p.Kp;
  }
  if (gx) {
    g.out = const_cast<void*>(grad_input->data);
    if (!run_product(p.type, LIN_DX, p.dx, g, partial, s)) return QMOE_ERR_HIP;
  }
  if (gw) {
    g.out = const_cast<void*>(grad_weights->data);
    if (!run_product(p.type, LIN_DW, p.dw, g, partial, s)) return QMOE_ERR_HIP;
  }
  return QMOE_OK;
}

}  // extern "C"
