// Host side of the norms around a block and their backward pass: validation,
// plans, launches; and their kernels' instantiations.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/gemm_preshuffle.h"
#include "host.hpp"
#include "norm.hpp"

namespace gp {
namespace {

constexpr int64_t kMaxGates = 256, kMaxRow = 16384;

// Waves of a row and 8-column pieces of a lane, and the workgroups.
struct NormPlan {
  int wpr = 1, c = 1;
  int64_t wgs = 1, per_gate = 1;   // per_gate: backward, of one gate row
};

bool norm_kind(int k) { return k >= GP_NORM_NONE && k <= GP_NORM_LAYER; }

int check_norm(int dtype, int64_t M, int64_t H, int64_t gates) {
  if (M <= 0 || H <= 0 || gates < 0) return GP_EINVAL;
  if (dtype != GP_BF16 && dtype != GP_F16) return GP_EDTYPE;
  if (M >= kMaxBytes || H % 8 || H > kMaxRow || gates > kMaxGates || (gates && M % gates)) return GP_ESHAPE;
  return GP_OK;
}

// One wave a row as long as it holds the row in 16 columns a lane (and there are rows
// for all waves), then the fewest waves that hold it in 8, and 16 from 4096 on. Measured us
// (residual add and RMS norm, graph of calls): 1 x 4096 on 8 waves of one piece 3.2, 4 of two
// 4.5, 16 of one 3.7; 1500 x 1024 on one wave of two 5.6, four of one 5.4, 16384 x 1024 26.1
// and 28.2; 3000 x 5120 on 8 of two 27.8, 16 of one 26.8, but with layer norms on both sides 37.8
// and 39.5; 4096 x 16384 on 16 of two 111, 8 of four 116.
void row_shape(int64_t M, int64_t H, NormPlan* p) {
  if (H <= 512) p->wpr = 1, p->c = 1;
  else if (H <= 1024 && M >= 1024) p->wpr = 1, p->c = 2;
  else if (H <= 2048) p->wpr = 4, p->c = 1;
  else if (H <= 4096) p->wpr = 8, p->c = 1;
  else if (H <= 8192) p->wpr = 8, p->c = 2;
  else p->wpr = 16, p->c = 2;
}

// The workgroups that the CUs hold at once (by their registers), or one per row (four
// rows of one wave each).
int64_t resident(const NormPlan& p) { return 256 * (p.wpr * p.c >= 16 ? 1 : p.wpr == 8 || p.c == 2 ? 2 : 4); }

NormPlan plan_norm(int64_t M, int64_t H) {
  NormPlan p;
  row_shape(M, H, &p);
  const int64_t rpw = norm_threads(p.wpr) / (64 * p.wpr);
  p.wgs = std::min(resident(p), (M + rpw - 1) / rpw);
  return p;
}

// Backward: fewer, since each workgroup writes its columns' sums, 16 bytes a column, and
// the next launch reads them, where a row's element takes 12 in all: one per CU of 8
// waves and more, two of fewer waves, and two of 8 where a norm_in's reductions want
// something beside them and the rows are many. Measured us (both launches, a norm_out
// alone unless named): 16384 x 4096 169 with 256 workgroups, 184 with 512; 2000 x 4096
// 26.0 and 31.2; with a norm_in 1500 x 4096 25.2 and 28.6, 2500 x 4096 33.4 and 34.7, 4000 x
// 3000 53.0 and 46.5; 16384 x 2048 with a norm_in 121 with 256, 82 with 512, 91 with 1024;
// 8192 x 512 15.1 with 512, 17.0 with 1024. Of those no more than share the rows evenly:
// 332 x 8680 23.3 with 166, 25.6 with 256. A workgroup stays within one gate row; where whole
// shares of the gate rows would leave a quarter of the CUs idle there is one more each.
NormPlan plan_norm_grad(int64_t M, int64_t H, int64_t gates, int norm_in) {
  NormPlan p;
  row_shape(M, H, &p);
  const int64_t rpw = norm_threads(p.wpr) / (64 * p.wpr), G = std::max<int64_t>(gates, 1);
  const int64_t per_cu = p.wpr < 8 || (p.wpr * p.c == 8 && norm_in != GP_NORM_NONE && M >= 3000) ? 2 : 1;
  const int64_t turns = (M / G + rpw - 1) / rpw;   // of one workgroup's, all rows of a gate row
  const int64_t cus = 256 * per_cu, whole = std::max<int64_t>(cus / G, 1);
  const int64_t most = whole * G < cus * 3 / 4 ? whole + 1 : whole, each = (turns + most - 1) / most;
  p.per_gate = (turns + each - 1) / each;
  p.wgs = G * p.per_gate;
  return p;
}

#define GP_NORM_SHAPES(X) X(1, 1) X(1, 2) X(4, 1) X(8, 1) X(8, 2) X(16, 2)

template <int DT>
hipError_t launch_norm(const NormPlan& p, const NormArgs& a, hipStream_t s) {
#define GP_NORM_CASE(W, C)                                                                              \
  if (p.wpr == W && p.c == C) {                                                                         \
    hipLaunchKernelGGL((norm_kernel<DT, W, C, (W * C < 32)>), dim3((uint32_t)p.wgs), dim3(norm_threads(W)), 0, s, a); \
    return hipGetLastError();                                                                           \
  }
  GP_NORM_SHAPES(GP_NORM_CASE)
#undef GP_NORM_CASE
  return hipErrorInvalidValue;
}

template <int DT, bool IN>
hipError_t launch_norm_grad(const NormPlan& p, const NormGradArgs& a, hipStream_t s) {
#define GP_NORM_CASE(W, C)                                                                                       \
  if (p.wpr == W && p.c == C) {                                                                                  \
    hipLaunchKernelGGL((norm_grad_kernel<DT, W, C, IN>), dim3((uint32_t)p.wgs), dim3(norm_threads(W)), 0, s, a); \
    return hipGetLastError();                                                                                    \
  }
  GP_NORM_SHAPES(GP_NORM_CASE)
#undef GP_NORM_CASE
  return hipErrorInvalidValue;
}

template <class... P>
bool aligned(const P*... p) { return (is_aligned16(p) && ...); }

}  // namespace
}  // namespace gp

using namespace gp;

extern "C" {

int gemm_norm(int dtype, const void* x, const void* residual, float scale, int norm_in, const float* w_in,
              const float* b_in, const float* gate, int64_t gates, int norm_out, const float* w_out,
              const float* b_out, float eps, void* r, void* y, int64_t M, int64_t H, void* stream) {
  if (!x || (!r && !y) || !norm_kind(norm_in) || !norm_kind(norm_out)) return GP_EINVAL;
  if (!gate != (gates == 0) || !y != (norm_out == GP_NORM_NONE) || !(eps >= 0.f)) return GP_EINVAL;
  if ((norm_in == GP_NORM_NONE && (w_in || b_in)) || (norm_out == GP_NORM_NONE && (w_out || b_out))) return GP_EINVAL;
  if (!aligned(x, residual, r, y) || !aligned(w_in, b_in, gate, w_out, b_out)) return GP_EINVAL;
  int e = check_norm(dtype, M, H, gates);
  if (e) return e;
  if ((e = require_gfx950())) return e;
  const NormPlan p = plan_norm(M, H);
  NormArgs a;
  a.x = (const char*)x;
  a.res = (const char*)residual;
  a.w_in = w_in;
  a.b_in = b_in;
  a.gate = gate;
  a.w_out = w_out;
  a.b_out = b_out;
  a.r = (char*)r;
  a.y = (char*)y;
  a.scale = scale;
  a.eps = eps;
  a.H = (uint32_t)H;
  a.gate_rows = (uint32_t)(gates ? M / gates : M);
  a.M = (uint64_t)M;
  a.kin = norm_in;
  a.kout = norm_out;
  forget_hip_error();
  const hipStream_t s = (hipStream_t)stream;
  return report_hip(dtype == GP_BF16 ? launch_norm<DT_BF16>(p, a, s) : launch_norm<DT_F16>(p, a, s), "kernel launch");
}

int gemm_norm_backward_workspace_size(int dtype, int64_t M, int64_t H, int64_t gates, size_t* bytes) {
  if (!bytes) return GP_EINVAL;
  const int e = check_norm(dtype, M, H, gates);
  if (e) return e;
  // (the most that any norm_in takes)
  *bytes = (size_t)(plan_norm_grad(M, H, gates, GP_NORM_RMS).wgs * 4 * H * 4);
  return GP_OK;
}

int gemm_norm_backward(int dtype, const void* dy, const void* dr, const void* x, const void* r, float scale,
                       int norm_in, const float* w_in, const float* b_in, const float* gate, int64_t gates,
                       int norm_out, const float* w_out, float eps, void* dx, void* dresidual, float* dw_in,
                       float* db_in, float* dgate, float* dw_out, float* db_out, int64_t M, int64_t H, void* workspace,
                       size_t workspace_bytes, void* stream) {
  const bool in = norm_in != GP_NORM_NONE, out = norm_out != GP_NORM_NONE;
  if (!norm_kind(norm_in) || !norm_kind(norm_out) || !gate != (gates == 0) || !(eps >= 0.f)) return GP_EINVAL;
  if (!dy != !out || (!dy && !dr)) return GP_EINVAL;
  if (!dx && !dresidual && !dw_in && !db_in && !dgate && !dw_out && !db_out) return GP_EINVAL;
  if (!in && (w_in || b_in || dw_in || db_in)) return GP_EINVAL;
  if (!out && (w_out || dw_out || db_out)) return GP_EINVAL;
  if (!gate && dgate) return GP_EINVAL;
  const bool use_x = (in && (dx || dw_in)) || dgate;
  if ((out && !r) || (use_x && !x)) return GP_EINVAL;
  if (!aligned(dy, dr, x, r, dx, dresidual, workspace) ||
      !aligned(w_in, b_in, gate, w_out, dw_in, db_in, dgate, dw_out, db_out))
    return GP_EINVAL;
  int e = check_norm(dtype, M, H, gates);
  if (e) return e;
  const NormPlan p = plan_norm_grad(M, H, gates, norm_in);
  const bool sums = dw_in || db_in || dgate || dw_out || db_out;
  if (sums && (!workspace || (int64_t)workspace_bytes < p.wgs * 4 * H * 4)) return GP_EWORKSPACE;
  if ((e = require_gfx950())) return e;
  NormGradArgs a;
  a.dy = (const char*)dy;
  a.dr = (const char*)dr;
  a.x = use_x ? (const char*)x : nullptr;
  a.r = (const char*)r;
  a.w_in = w_in;
  a.gate = gate;
  a.w_out = w_out;
  a.dx = (char*)dx;
  a.dres = (char*)dresidual;
  a.part = (float*)workspace;
  a.scale = scale;
  a.eps = eps;
  a.H = (uint32_t)H;
  a.gate_rows = (uint32_t)(gates ? M / gates : M);
  a.wgs_per_gate = (uint32_t)p.per_gate;
  a.sums = (dw_out ? 1u : 0u) | (db_out ? 2u : 0u) | (dw_in || dgate ? 4u : 0u) | (db_in || (dgate && b_in) ? 8u : 0u);
  a.kin = norm_in;
  a.kout = norm_out;
  forget_hip_error();
  const hipStream_t s = (hipStream_t)stream;
  auto* launch = in || gate ? (dtype == GP_BF16 ? launch_norm_grad<DT_BF16, true> : launch_norm_grad<DT_F16, true>)
                            : (dtype == GP_BF16 ? launch_norm_grad<DT_BF16, false> : launch_norm_grad<DT_F16, false>);
  e = report_hip(launch(p, a, s), "kernel launch");
  if (e || !sums) return e;
  NormSumsArgs t;
  t.part = (const float*)workspace;
  t.gate = gate;
  t.w_in = w_in;
  t.b_in = b_in;
  t.dw_out = dw_out;
  t.db_out = db_out;
  t.dw_in = dw_in;
  t.db_in = db_in;
  t.dgate = dgate;
  t.H = (uint32_t)H;
  t.parts = (uint32_t)p.wgs;
  t.wgs_per_gate = (uint32_t)p.per_gate;
  forget_hip_error();
  hipLaunchKernelGGL(norm_sums_kernel, dim3((uint32_t)((H + 63) / 64), (uint32_t)(4 + gates)), dim3(1024), 0, s, t);
  return report_hip(hipGetLastError(), "kernel launch");
}

}  // extern "C"
