// Host side of the mixture-of-experts layer for a few tokens: validation, plan,
// workspace, launches; and its kernels' instantiations.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gemm_preshuffle.h"
#include "host.hpp"
#include "moe.hpp"

namespace gp {
namespace {

constexpr int64_t kMaxTokens = 256, kMaxChoices = 32;

int64_t whole_k(int64_t K) { return (K + 63) / 64 * 64; }
int64_t up_bytes(int64_t F, int64_t H) { return 4 * F * whole_k(H); }     // of one expert
int64_t down_bytes(int64_t F, int64_t H) { return 2 * H * whole_k(F); }
int64_t align256(int64_t v) { return (v + 255) & ~(int64_t)255; }

// 16-byte pieces of the experts' layouts (as preshuffle_ffn_kernel's), an expert per
// blockIdx.y
__global__ __launch_bounds__(256) void preshuffle_experts_kernel(const char* __restrict__ w, char* __restrict__ dst,
                                                                 uint32_t kb64, uint32_t Ka, uint32_t F, uint32_t chunks,
                                                                 size_t from_bytes) {
  const uint32_t x = blockIdx.x * 256u + threadIdx.x;
  if (x >= chunks) return;
  const uint32_t j = x & 15u, g = (x >> 4) & 3u, t = x >> 6;
  const uint32_t k0 = t % kb64, nb = t / kb64;
  const uint32_t row = (F ? (nb & 1u) * F + (nb >> 1) * 16u : nb * 16u) + j, col = 64u * k0 + 16u * g;
  const char* src = w + blockIdx.y * from_bytes;
  *(v4i*)(dst + (blockIdx.y * (size_t)chunks + x) * 16u) = col < Ka ? *(const v4i*)(src + (size_t)row * Ka + col) : v4i{0, 0, 0, 0};
}

int check_weights(int dtype, int64_t E, int64_t F, int64_t H) {
  if (E <= 0 || F <= 0 || H <= 0) return GP_EINVAL;
  if (dtype != GP_BF16 && dtype != GP_F16) return GP_EDTYPE;
  if (E > kMaxExperts || F >= kMaxBytes / 4 || H >= kMaxBytes / 4 || F % 16 || H % 32) return GP_ESHAPE;
  if (!fits(2 * F, 2 * whole_k(H)) || !fits(H, 2 * whole_k(F))) return GP_ESHAPE;
  return GP_OK;
}

// Workspace: 64 KiB of arrival counters (a column group of the down product each, the
// router's token blocks in the last 256), the logits, the pairs' h, their products.
struct MoePlan {
  int xl = 0;                      // rows at a time: 1, or 8 xl
  int64_t slots = 0, up_cols = 0, down_cols = 0;
  int64_t off_logits = 0, off_h = 0, off_part = 0, bytes = 0;
};
constexpr int64_t kRouteCounters = 256;

int plan_moe(int dtype, int64_t M, int64_t F, int64_t H, int64_t E, int64_t k, MoePlan* p) {
  if (M <= 0 || k <= 0) return GP_EINVAL;
  const int r = check_weights(dtype, E, F, H);
  if (r) return r;
  if (M > kMaxTokens || k > E || k > kMaxChoices || M * k > kMaxPairs) return GP_ESHAPE;
  if (H / 16 > kMaxSplitTiles - kRouteCounters || !fits(M * k, 4 * H) || !fits(M * k, 2 * F)) return GP_ESHAPE;
  // rows at a time for the longest list of an expert, about twice the average (further
  // turns read the weights again, mostly from L2)
  const int64_t most = M * k / E;
  p->xl = M == 1 ? 0 : M <= 8 || most <= 3 ? 1 : M <= 16 || most <= 14 ? 2 : most <= 30 ? 4 : 8;
  p->slots = std::min(M * k, E);
  p->up_cols = F / 16;
  p->down_cols = p->xl == 0 ? H / 16 : (H / 16 + 1) / 2;
  p->off_logits = kCounterBytes;
  p->off_h = p->off_logits + align256(M * E * 8);
  p->off_part = p->off_h + align256(M * k * F * 2);
  p->bytes = p->off_part + align256(M * k * H * 4);
  if (p->slots * std::max(p->up_cols, p->down_cols) >= (int64_t)1 << 22) return GP_ESHAPE;   // threads of a grid
  return GP_OK;
}

// Variants: rows, 16-column blocks, waves, chunks of K in flight per group. Measured us
// (both products, up's or down's variant alone changed), M, k of E, H x F:
//   16, 8 of 64, 2048 x 1024: up 8 rows on 8 waves 143, 16 rows on 4 of one chunk 145, of two
//     chunks on 8 159; down two blocks on 4 waves 135, one on 8 159 (8192 workgroups of 32 KB)
//   64, 8 of 128, 2048 x 768: up 16 rows 312, 8 rows 319 (longest list 11), with 8 waves and two
//     chunks 359; down two blocks on 4 waves 256, one on 8 359
//   64, 2 of 4, 2048 x 4096: up 64 rows 67, 32 rows 75, 16 rows 97 (longest list 39)
//   33, 2 of 8, 4096 x 14336: up 16 rows 452, 32 rows 458; down two blocks on 8 waves 462, one 470
//   one token, 8 of 64, 2048 x 1024: up 8 waves of two chunks 20.8, 4 of four 21.4; down 8 waves
//     20.8, 16 20.8, as the general form 23.7
#define GP_MOE_CASE(XL, NB, W, S, UP)                                                                            \
  if (xl == XL && up == UP) {                                                                                    \
    hipLaunchKernelGGL((moe_kernel<DT, XL, NB, W, S, UP>), dim3(a.slots * a.cols), dim3(W * 64), 0, s, a);       \
    return hipGetLastError();                                                                                    \
  }
template <int DT>
hipError_t launch_moe(int xl, bool up, const MoeArgs& a, hipStream_t s) {
  GP_MOE_CASE(0, 2, 8, 2, true)
  GP_MOE_CASE(1, 2, 8, 1, true)
  GP_MOE_CASE(2, 2, 4, 1, true)
  GP_MOE_CASE(4, 2, 4, 1, true)
  GP_MOE_CASE(8, 2, 4, 1, true)
  if (xl == 0) {
    hipLaunchKernelGGL((moe_down_one_kernel<DT, 1, 8, 2>), dim3(a.cols), dim3(512), 0, s, a);
    return hipGetLastError();
  }
  GP_MOE_CASE(1, 2, 4, 1, false)
  GP_MOE_CASE(2, 2, 4, 1, false)
  GP_MOE_CASE(4, 2, 8, 1, false)
  GP_MOE_CASE(8, 2, 8, 1, false)
  return hipErrorInvalidValue;
}
#undef GP_MOE_CASE

template <int DT>
hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  // tokens and experts of a workgroup
  if (a.M == 1) hipLaunchKernelGGL((route_kernel<DT, 1, 4>), dim3((a.E + 3) / 4, 1), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((route_kernel<DT, 4, 4>), dim3((a.E + 3) / 4, (a.M + 3) / 4), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <class... P>
bool aligned(const P*... p) { return (is_aligned16(p) && ...); }

int run_route(int dtype, const void* x, const void* router, const float* bias, int score, int normalize, float scale,
              int32_t* ids, float* gates, int64_t M, int64_t H, int64_t E, int64_t k, const MoePlan& p, char* ws,
              hipStream_t s) {
  RouteArgs a;
  a.x = (const char*)x;
  a.wr = (const char*)router;
  a.bias = bias;
  a.logits = (double*)(ws + p.off_logits);
  a.cnt = (uint32_t*)ws + (kMaxSplitTiles - kRouteCounters);
  a.ids = ids;
  a.gates = gates;
  a.M = (uint32_t)M;
  a.E = (uint32_t)E;
  a.H = (uint32_t)H;
  a.k = (uint32_t)k;
  a.sigmoid = score == GP_SCORE_SIGMOID;
  a.normalize = normalize != 0;
  a.scale = scale;
  forget_hip_error();
  return report_hip(dtype == GP_BF16 ? launch_route<DT_BF16>(a, s) : launch_route<DT_F16>(a, s), "kernel launch");
}

int run_experts(int dtype, const void* x, const void* w_shuf, const int32_t* ids, const float* gates, int act,
                const void* residual, void* y, int64_t M, int64_t F, int64_t H, int64_t E, int64_t k, const MoePlan& p,
                char* ws, hipStream_t s) {
  MoeArgs a = {};
  a.ids = ids;
  a.gates = gates;
  a.cnt = (uint32_t*)ws;
  a.M = (uint32_t)M;
  a.k = (uint32_t)k;
  a.E = (uint32_t)E;
  a.slots = (uint32_t)p.slots;
  a.act = act;
  a.h = ws + p.off_h;
  a.a = (const char*)x;
  a.b = (const char*)w_shuf;
  a.expert_bytes = (size_t)up_bytes(F, H);
  a.F = (uint32_t)F;
  a.Ka = (uint32_t)(2 * H);
  a.Kb = (uint32_t)(2 * whole_k(H));
  a.cols = (uint32_t)p.up_cols;
  const bool bf16 = dtype == GP_BF16;
  forget_hip_error();
  const int r = report_hip(bf16 ? launch_moe<DT_BF16>(p.xl, true, a, s) : launch_moe<DT_F16>(p.xl, true, a, s), "kernel launch");
  if (r) return r;
  a.a = a.h;
  a.b = (const char*)w_shuf + E * up_bytes(F, H);
  a.expert_bytes = (size_t)down_bytes(F, H);
  a.res = (const char*)residual;
  a.y = (char*)y;
  a.part = (float*)(ws + p.off_part);
  a.F = (uint32_t)H;
  a.Ka = (uint32_t)(2 * F);
  a.Kb = (uint32_t)(2 * whole_k(F));
  a.cols = (uint32_t)p.down_cols;
  forget_hip_error();
  return report_hip(bf16 ? launch_moe<DT_BF16>(p.xl, false, a, s) : launch_moe<DT_F16>(p.xl, false, a, s), "kernel launch");
}

int check_route(const void* x, const void* router, const float* bias, int score, int32_t* ids, float* gates) {
  if (!x || !router || !ids || !gates || !aligned(x, router) || !aligned(bias, gates) || !is_aligned16(ids)) return GP_EINVAL;
  return score == GP_SCORE_SOFTMAX || score == GP_SCORE_SIGMOID ? GP_OK : GP_EINVAL;
}
int check_experts(const void* x, const void* w_shuf, const int32_t* ids, const float* gates, int act,
                  const void* residual, void* y) {
  if (!x || !w_shuf || !ids || !gates || !y || !aligned(x, w_shuf, residual, y) || !is_aligned16(ids) || !is_aligned16(gates))
    return GP_EINVAL;
  return act < GP_ACT_NONE || act > GP_ACT_GELU ? GP_EINVAL : GP_OK;
}
int check_workspace(const MoePlan& p, void* workspace, size_t workspace_bytes) {
  if (!workspace || (int64_t)workspace_bytes < p.bytes) return GP_EWORKSPACE;
  return is_aligned16(workspace) ? GP_OK : GP_EINVAL;
}

}  // namespace
}  // namespace gp

using namespace gp;

extern "C" {

int gemm_moe_weights_size(int64_t E, int64_t F, int64_t H, size_t* bytes) {
  if (!bytes) return GP_EINVAL;
  const int r = check_weights(GP_BF16, E, F, H);
  if (r) return r;
  *bytes = (size_t)(E * (up_bytes(F, H) + down_bytes(F, H)));
  return GP_OK;
}

int gemm_moe_preshuffle(int dtype, const void* w13, const void* w2, void* w_shuf, int64_t E, int64_t F, int64_t H,
                        void* stream) {
  if (!w13 || !w2 || !w_shuf || !aligned(w13, w2, w_shuf)) return GP_EINVAL;
  int r = check_weights(dtype, E, F, H);
  if (r) return r;
  const int64_t up = up_bytes(F, H), down = down_bytes(F, H);
  const char *s = (const char*)w_shuf, *end = s + E * (up + down), *a = (const char*)w13, *b = (const char*)w2;
  if ((s < a + E * 4 * F * H && a < end) || (s < b + E * 2 * F * H && b < end)) return GP_EINVAL;   // overlap
  if ((r = require_gfx950())) return r;
  const hipStream_t q = (hipStream_t)stream;
  forget_hip_error();
  hipLaunchKernelGGL(preshuffle_experts_kernel, dim3((uint32_t)((up / 16 + 255) / 256), (uint32_t)E), dim3(256), 0, q, a,
                     (char*)w_shuf, (uint32_t)(whole_k(H) / 32), (uint32_t)(2 * H), (uint32_t)F, (uint32_t)(up / 16),
                     (size_t)(4 * F * H));
  if ((r = report_hip(hipGetLastError(), "kernel launch"))) return r;
  forget_hip_error();
  hipLaunchKernelGGL(preshuffle_experts_kernel, dim3((uint32_t)((down / 16 + 255) / 256), (uint32_t)E), dim3(256), 0, q, b,
                     (char*)w_shuf + E * up, (uint32_t)(whole_k(F) / 32), (uint32_t)(2 * F), 0u, (uint32_t)(down / 16),
                     (size_t)(2 * F * H));
  return report_hip(hipGetLastError(), "kernel launch");
}

int gemm_moe_workspace_size(int dtype, int64_t M, int64_t F, int64_t H, int64_t E, int64_t k, size_t* bytes) {
  if (!bytes) return GP_EINVAL;
  MoePlan p;
  const int r = plan_moe(dtype, M, F, H, E, k, &p);
  if (r) return r;
  *bytes = (size_t)p.bytes;
  return GP_OK;
}

int gemm_moe_route(int dtype, const void* x, const void* router, const float* bias, int score, int normalize, float scale,
                   int32_t* ids, float* gates, int64_t M, int64_t H, int64_t E, int64_t k, void* workspace,
                   size_t workspace_bytes, void* stream) {
  int r = check_route(x, router, bias, score, ids, gates);
  if (r) return r;
  MoePlan p;
  if ((r = plan_moe(dtype, M, 16, H, E, k, &p))) return r;
  // (only the counters and the logits of the layer's workspace)
  if (!workspace || (int64_t)workspace_bytes < p.off_h) return GP_EWORKSPACE;
  if (!is_aligned16(workspace)) return GP_EINVAL;
  if ((r = require_gfx950())) return r;
  return run_route(dtype, x, router, bias, score, normalize, scale, ids, gates, M, H, E, k, p, (char*)workspace,
                   (hipStream_t)stream);
}

int gemm_moe_experts(int dtype, const void* x, const void* w_shuf, const int32_t* ids, const float* gates, int act,
                     const void* residual, void* y, int64_t M, int64_t F, int64_t H, int64_t E, int64_t k,
                     void* workspace, size_t workspace_bytes, void* stream) {
  int r = check_experts(x, w_shuf, ids, gates, act, residual, y);
  if (r) return r;
  MoePlan p;
  if ((r = plan_moe(dtype, M, F, H, E, k, &p)) || (r = check_workspace(p, workspace, workspace_bytes))) return r;
  if ((r = require_gfx950())) return r;
  return run_experts(dtype, x, w_shuf, ids, gates, act, residual, y, M, F, H, E, k, p, (char*)workspace, (hipStream_t)stream);
}

int gemm_moe(int dtype, const void* x, const void* router, const float* bias, int score, int normalize, float scale,
             const void* w_shuf, int act, const void* residual, void* y, int32_t* ids, float* gates, int64_t M, int64_t F,
             int64_t H, int64_t E, int64_t k, void* workspace, size_t workspace_bytes, void* stream) {
  int r = check_route(x, router, bias, score, ids, gates);
  if (r || (r = check_experts(x, w_shuf, ids, gates, act, residual, y))) return r;
  MoePlan p;
  if ((r = plan_moe(dtype, M, F, H, E, k, &p)) || (r = check_workspace(p, workspace, workspace_bytes))) return r;
  if ((r = require_gfx950())) return r;
  char* ws = (char*)workspace;
  const hipStream_t s = (hipStream_t)stream;
  if ((r = run_route(dtype, x, router, bias, score, normalize, scale, ids, gates, M, H, E, k, p, ws, s))) return r;
  return run_experts(dtype, x, w_shuf, ids, gates, act, residual, y, M, F, H, E, k, p, ws, s);
}

}  // extern "C"
