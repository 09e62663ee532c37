// Host side of the products with 4-bit weights and group scales: validation,
// layout, plan, launch.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gemm_preshuffle.h"
#include "host.hpp"
#include "launch_w4.hpp"

namespace gp {
namespace {

// Laid-out weights: blocks, then scales, then zero points, each 256-aligned.
struct W4Layout {
  int64_t nblk = 0, kblk = 0, sblk = 0;
  int sg = 1, sshift = 0;
  int64_t off_s = 0, off_z = 0, bytes = 0;
};

int64_t align256(int64_t v) { return (v + 255) & ~(int64_t)255; }

// N: rows of the weights (gated: 2 F). One workgroup's rows of x and blocks of
// weights are addressed with 32-bit offsets (K below 2^23); everything else is
// 64-bit.
int layout_w4(int64_t N, int64_t K, int group, bool zeros, bool gated, W4Layout* l) {
  if (N <= 0 || K <= 0 || group <= 0) return GP_EINVAL;
  if (N >= kMaxBytes || K >= (int64_t)1 << 23 || K % 32 || group < 32 || (group & (group - 1))) return GP_ESHAPE;
  if (gated && N % 2) return GP_ESHAPE;
  l->nblk = gated ? 2 * ((N / 2 + 15) / 16) : (N + 15) / 16;
  l->kblk = (K + 127) / 128;
  l->sg = group >= 128 ? 1 : 128 / group;
  l->sshift = 0;
  while (l->sshift < 20 && ((int64_t)256 << l->sshift) <= group) ++l->sshift;
  l->sblk = (l->kblk + ((int64_t)1 << l->sshift) - 1) >> l->sshift;
  const int64_t entries = l->nblk * l->sblk * 16 * l->sg;
  l->off_s = l->nblk * l->kblk * 1024;
  l->off_z = l->off_s + align256(entries * 2);
  l->bytes = l->off_z + (zeros ? align256(entries) : 0);
  // one thread per 16 bytes of the layout
  if (l->nblk * l->kblk * 64 >= (int64_t)1 << 32) return GP_ESHAPE;
  return GP_OK;
}

struct W4LayoutArgs {
  const uint8_t* q;
  const uint16_t* scales;
  const int8_t* zeros;
  char *w, *s, *z;
  uint32_t N, K, group, groups, F;   // F: 0, or gate rows of a gated matrix
  uint32_t nblk, kblk, sblk, sg;
};

// Row of the weights in column j of block nb; N if there is none.
__device__ __forceinline__ uint32_t w4_row(const W4LayoutArgs& p, uint32_t nb, uint32_t j) {
  if (!p.F) return min(nb * 16 + j, p.N);
  const uint32_t f = nb / 2 * 16 + j;
  return f < p.F ? (nb & 1u) * p.F + f : p.N;
}

// One thread per 16 bytes of weights; the first of them also write the scales
// and zero points.
__global__ __launch_bounds__(256) void layout_w4_kernel(W4LayoutArgs p) {
  const uint64_t x = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  const uint64_t pieces = (uint64_t)p.nblk * p.kblk * 64;
  if (x < pieces) {
    const uint32_t j = x & 15, hi = (x >> 4) & 3, b = (uint32_t)((x >> 6) % p.kblk), nb = (uint32_t)((x >> 6) / p.kblk);
    const uint32_t row = w4_row(p, nb, j);
    v4i o;
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      const uint32_t k = b * 128 + st * 32 + hi * 8;
      uint32_t d = 0;   // eight nibbles, two's complement; absent ones are 0
      if (row < p.N && k < p.K) d = *(const uint32_t*)(p.q + ((size_t)row * p.K + k) / 2);
      uint32_t v = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) v |= ((d >> (4 * i)) & 15u) << (i < 4 ? 8 * i : 8 * (i - 4) + 4);
      o[st] = (int)(v ^ 0x88888888u);
    }
    *(v4i*)(p.w + x * 16) = o;
  }
  const uint64_t entries = (uint64_t)p.nblk * p.sblk * 16 * p.sg;
  if (x < entries) {
    const uint32_t g = x % p.sg, j = x / p.sg % 16, sb = (uint32_t)(x / p.sg / 16 % p.sblk),
                   nb = (uint32_t)(x / p.sg / 16 / p.sblk);
    const uint32_t row = w4_row(p, nb, j), grp = sb * p.sg + g;
    const bool on = row < p.N && grp < p.groups;
    ((uint16_t*)p.s)[x] = on ? p.scales[(size_t)row * p.groups + grp] : (uint16_t)0;
    if (p.z) ((int8_t*)p.z)[x] = on ? p.zeros[(size_t)row * p.groups + grp] : (int8_t)0;
  }
}

// The variant by the number of rows and column blocks; microseconds on one
// MI355X, groups of 128 unless named (nb x waves, chunks of one K block):
//   one row, up to 4 rows: 16 waves on single blocks while those give at most
//     two workgroups per CU: 4096 x 4096 3.95 (8 waves 4.53, pairs 4.24), 8192 x
//     28672 22.7 (pairs on 8 waves 23.0); above, pairs on 8 waves: 28672 x 8192
//     21.4 (21.7), and on 4 waves with chunks of two where 8 would have less
//     than four K blocks each: 32768 x 2048 8.4 (9.4 on 8 waves, 11.8 on 16);
//     3 rows, gated, 14336 x 4096 14.1 on fours and 4 waves (pairs on 8 14.5).
//   more rows: as many blocks per workgroup as still give one workgroup per CU,
//     since every workgroup reads all of x: 16 rows 16384 x 8192 15.3 on fours
//     (pairs 18.8, single 25.5), 4091 x 7168 in groups of 64 8.0 on single ones
//     (pairs 9.5); 32 rows 14336 x 8192 19.0 on fours (25.9, 40.9), 4096 x 4096
//     7.6 on single ones (8.7); 64 rows 14336 x 8192 33.9 on fours (46.5).
// split: with a workspace, K is split where few column blocks leave CUs idle.
struct W4Split { int64_t tiles = 0, ks = 1, bytes = 0; };
int plan_w4(int64_t M, const W4Layout& l, bool gated, bool split, W4Plan* p, W4Split* k) {
  p->xl = M == 1 ? 0 : M <= 4 ? 1 : M <= 16 ? 4 : M <= 32 ? 8 : 16;
  if (p->xl <= 1) {
    const bool many = l.nblk > 512;
    p->nb = gated || many ? 2 : 1;
    p->waves = many ? 8 : 16;
    if (many && p->xl == 1) {
      p->nb = 4;
      p->waves = 4;
    } else if (many && l.kblk < 32) {
      p->waves = 4;
      p->s = 2;
    }
  } else {
    p->nb = l.nblk >= 1024 || (p->xl > 4 && l.nblk >= 768) ? 4 : gated || l.nblk >= 512 ? 2 : 1;
    p->waves = p->xl == 16 && p->nb > 1 ? 4 : 8;
  }
  const int64_t rows = p->xl == 0 ? 1 : 4 * p->xl;
  const int64_t wgs = ((l.nblk + p->nb - 1) / p->nb) * ((M + rows - 1) / rows);
  if (wgs * p->waves * 64 >= (int64_t)1 << 32) return GP_ESHAPE;
  k->tiles = wgs;
  if (split) {
    const double step_us = p->xl <= 1 ? 0.45 : p->xl == 4 ? 0.55 : p->xl == 8 ? 1.0 : 1.9;
    k->ks = split_small((double)l.kblk / p->waves, step_us, wgs);
    if (k->ks > 1) k->bytes = kCounterBytes + wgs * k->ks * ((rows + 15) / 16 * p->nb * (p->xl == 0 ? 256 : 1024));
  }
  return GP_OK;
}

int run_w4(int dtype, const void* x, const void* w_shuf, bool zeros, const float* bias, int act, void* y, int64_t M,
           int64_t N, int64_t K, int group, bool gated, bool split, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!x || !w_shuf || !y || !is_aligned16(x) || !is_aligned16(w_shuf) || !is_aligned16(y) || !is_aligned16(bias))
    return GP_EINVAL;
  if (M <= 0 || act < GP_ACT_NONE || act > GP_ACT_GELU) return GP_EINVAL;
  if (dtype != GP_BF16 && dtype != GP_F16) return GP_EDTYPE;
  if (M >= kMaxBytes || N >= kMaxBytes / 2) return GP_ESHAPE;
  W4Layout l;
  int r = layout_w4(gated ? 2 * N : N, K, group, zeros, gated, &l);
  if (r) return r;
  W4Plan p;
  W4Split k;
  if ((r = plan_w4(M, l, gated, split, &p, &k))) return r;
  if (k.ks > 1) {
    if (!ws || (int64_t)ws_bytes < k.bytes) return GP_EWORKSPACE;
    if (!is_aligned16(ws)) return GP_EINVAL;
  }
  if ((r = require_gfx950())) return r;
  W4Args a;
  a.x = (const char*)x;
  a.w = (const char*)w_shuf;
  a.s = a.w + l.off_s;
  a.z = zeros ? a.w + l.off_z : nullptr;
  a.bias = bias;
  a.y = (char*)y;
  a.M = (uint32_t)M;
  a.N = (uint32_t)N;
  a.K = (uint32_t)K;
  a.nblk = (uint32_t)l.nblk;
  a.sshift = (uint32_t)l.sshift;
  a.act = act;
  a.gated = gated ? 1 : 0;
  a.ksplit = (uint32_t)k.ks;
  a.cnt = k.ks > 1 ? (uint32_t*)ws : nullptr;
  a.part = k.ks > 1 ? (char*)ws + kCounterBytes : nullptr;
  forget_hip_error();
  auto* launch = dtype == GP_BF16 ? (zeros ? launch_w4_bf16_z : launch_w4_bf16) : (zeros ? launch_w4_f16_z : launch_w4_f16);
  return report_hip(launch(p, l.sg, a, stream), "kernel launch");
}

}  // namespace
}  // namespace gp

using namespace gp;

extern "C" {

int gemm_w4a16_weights_size(int64_t N, int64_t K, int group, int has_zeros, int gated, size_t* bytes) {
  if (!bytes) return GP_EINVAL;
  W4Layout l;
  const int r = layout_w4(N, K, group, has_zeros != 0, gated != 0, &l);
  if (r) return r;
  *bytes = (size_t)l.bytes;
  return GP_OK;
}

int gemm_w4a16_preshuffle(int dtype, const void* q, const void* scales, const int8_t* zeros, void* w_shuf, int64_t N,
                          int64_t K, int group, int gated, void* stream) {
  if (!q || !scales || !w_shuf || !is_aligned16(q) || !is_aligned16(scales) || !is_aligned16(zeros) ||
      !is_aligned16(w_shuf))
    return GP_EINVAL;
  if (dtype != GP_BF16 && dtype != GP_F16) return GP_EDTYPE;
  W4Layout l;
  int r = layout_w4(N, K, group, zeros != nullptr, gated != 0, &l);
  if (r) return r;
  const int64_t groups = (K + group - 1) / group;
  auto overlap = [&](const void* src, int64_t bytes) {
    const char *a = (const char*)src, *b = (const char*)w_shuf;
    return src && a < b + l.bytes && b < a + bytes;
  };
  if (overlap(q, N * K / 2) || overlap(scales, N * groups * 2) || overlap(zeros, N * groups)) return GP_EINVAL;
  if ((r = require_gfx950())) return r;
  W4LayoutArgs a;
  a.q = (const uint8_t*)q;
  a.scales = (const uint16_t*)scales;
  a.zeros = zeros;
  a.w = (char*)w_shuf;
  a.s = a.w + l.off_s;
  a.z = zeros ? a.w + l.off_z : nullptr;
  a.N = (uint32_t)N;
  a.K = (uint32_t)K;
  a.group = (uint32_t)group;
  a.groups = (uint32_t)groups;
  a.F = gated ? (uint32_t)(N / 2) : 0u;
  a.nblk = (uint32_t)l.nblk;
  a.kblk = (uint32_t)l.kblk;
  a.sblk = (uint32_t)l.sblk;
  a.sg = (uint32_t)l.sg;
  // a 128-element block has at most 64 scales, one per 16-byte piece of it
  const int64_t threads = l.nblk * l.kblk * 64;
  forget_hip_error();
  hipLaunchKernelGGL(layout_w4_kernel, dim3((uint32_t)((threads + 255) / 256)), dim3(256), 0, (hipStream_t)stream, a);
  return report_hip(hipGetLastError(), "kernel launch");
}

int gemm_w4a16(int dtype, const void* x, const void* w_shuf, int has_zeros, const float* bias, int act, void* y,
               int64_t M, int64_t N, int64_t K, int group, void* stream) {
  return run_w4(dtype, x, w_shuf, has_zeros != 0, bias, act, y, M, N, K, group, false, false, nullptr, 0,
                (hipStream_t)stream);
}

int gemm_w4a16_gated(int dtype, const void* x, const void* w_shuf, int has_zeros, int act, void* h, int64_t M,
                     int64_t F, int64_t K, int group, void* stream) {
  return run_w4(dtype, x, w_shuf, has_zeros != 0, nullptr, act, h, M, F, K, group, true, false, nullptr, 0,
                (hipStream_t)stream);
}

int gemm_w4a16_workspace_size(int64_t M, int64_t N, int64_t K, int group, int gated, size_t* bytes) {
  if (!bytes || M <= 0) return GP_EINVAL;
  if (M >= kMaxBytes || N >= kMaxBytes / 2) return GP_ESHAPE;
  W4Layout l;
  int r = layout_w4(gated ? 2 * N : N, K, group, false, gated != 0, &l);
  if (r) return r;
  W4Plan p;
  W4Split k;
  if ((r = plan_w4(M, l, gated != 0, true, &p, &k))) return r;
  *bytes = (size_t)k.bytes;
  return GP_OK;
}

int gemm_w4a16_plan(int64_t M, int64_t N, int64_t K, int group, int gated, int with_workspace, gemm_plan_info* out) {
  if (!out || M <= 0) return GP_EINVAL;
  if (M >= kMaxBytes || N >= kMaxBytes / 2) return GP_ESHAPE;
  W4Layout l;
  int r = layout_w4(gated ? 2 * N : N, K, group, false, gated != 0, &l);
  if (r) return r;
  W4Plan p;
  W4Split k;
  if ((r = plan_w4(M, l, gated != 0, with_workspace != 0, &p, &k))) return r;
  *out = gemm_plan_info();
  out->kernel = GP_KERNEL_SPLITK;
  out->tile_m = p.xl == 0 ? 1 : 4 * p.xl;
  out->tile_n = 16 * p.nb;
  out->tile_k = 128 * p.s;
  out->waves = p.waves;
  out->threads = 64 * p.waves;
  out->ksplit = (int)k.ks;
  out->grid = k.tiles * k.ks;
  out->mfma = 16;
  out->workspace_bytes = k.bytes;
  return GP_OK;
}

int gemm_w4a16_ws(int dtype, const void* x, const void* w_shuf, int has_zeros, const float* bias, int act, void* y,
                  int64_t M, int64_t N, int64_t K, int group, int gated, void* workspace, size_t workspace_bytes,
                  void* stream) {
  if (gated && bias) return GP_EINVAL;
  return run_w4(dtype, x, w_shuf, has_zeros != 0, bias, act, y, M, N, K, group, gated != 0, true, workspace,
                workspace_bytes, (hipStream_t)stream);
}

}  // extern "C"
