// Transposing passes over 16-bit matrices, for the products whose K axis is
// the slow axis of an operand (the backward pass), and the gated block's
// pointwise backward, which writes its results both ways. All are bound by
// HBM: each element is read once and written once per layout.
//
// One workgroup of 256 threads moves a 64 x 64 tile through LDS. A thread
// loads 16 bytes (8 columns) of two adjacent rows and writes them as 8 dwords
// of one row pair each, so LDS holds the tile transposed, [column][row pair].
// Rows of 36 dwords keep 16-byte reads aligned; the row pair index is XORed
// with 8 * (column / 16), which gives the 64 lanes of a write 64 different
// banks (8 column groups of 8 would otherwise meet in two groups of 32).
#pragma once

#include "gp_common.hpp"

namespace gp {

constexpr int kTileLd = 36;   // dwords per transposed row

struct Tile64 {
  uint32_t d[64 * kTileLd];
  // rows 2 rp and 2 rp + 1 of columns 8 q .. 8 q + 7
  __device__ __forceinline__ void put(int q, int rp, v4i r0, v4i r1) {
    const int at = (8 * q) * kTileLd + (rp ^ ((q >> 1) << 3));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d[at + (2 * i) * kTileLd] = __builtin_amdgcn_perm((uint32_t)r1[i], (uint32_t)r0[i], 0x05040100u);
      d[at + (2 * i + 1) * kTileLd] = __builtin_amdgcn_perm((uint32_t)r1[i], (uint32_t)r0[i], 0x07060302u);
    }
  }
  // rows 8 g .. 8 g + 7 of column c
  __device__ __forceinline__ v4i get(int c, int g) const {
    return *(const v4i*)(d + c * kTileLd + ((4 * g) ^ ((c >> 4) << 3)));
  }
};

// the transposed tile as rows c0 .. c0 + 63 of dst [C][Kp], columns r0 .. r0 + 63
__device__ __forceinline__ void store_transposed(const Tile64& t, char* dst, uint32_t c0, uint32_t r0, uint32_t C,
                                                 uint32_t Kp) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int x = i * 256 + threadIdx.x;
    const int g = x & 7, c = x >> 3;
    if (c0 + c >= C || r0 + 8 * g >= Kp) continue;
    *(v4i*)(dst + ((size_t)(c0 + c) * Kp + r0 + 8 * g) * 2) = t.get(c, g);
  }
}

// A transposed copy of src [R][C] (C % 16 == 0), rows from R to Kp (a multiple
// of 32) taken as zeros: dst [C][Kp], or (preshuffled) the layout of B = src^T,
// B[n = c][k = r].
struct CopyJob {
  const char* src;
  char* dst;
  uint32_t R, C, Kp, tiles_c, blocks;   // 64 x 64 tiles per row of tiles, and in all
  uint32_t preshuffled;
};
__device__ __forceinline__ void copy_tile(Tile64& t, const CopyJob& p, uint32_t block) {
  const uint32_t c0 = block % p.tiles_c * 64u, r0 = block / p.tiles_c * 64u;
  const int q = threadIdx.x & 7, rp = threadIdx.x >> 3;
  const uint32_t r = r0 + 2 * rp, c = c0 + 8 * q;
  v4i a = v4i{0, 0, 0, 0}, b = a;
  if (c < p.C) {
    const char* s = p.src + ((size_t)r * p.C + c) * 2;
    if (r < p.R) a = *(const v4i*)s;
    if (r + 1 < p.R) b = *(const v4i*)(s + (size_t)p.C * 2);
  }
  t.put(q, rp, a, b);
  __syncthreads();
  if (!p.preshuffled) {
    store_transposed(t, p.dst, c0, r0, p.C, p.Kp);
    return;
  }
  // chunk (16-column block nb, 32-row block kb, group g, column j) of the tile
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int x = i * 256 + threadIdx.x;
    const int j = x & 15, g = (x >> 4) & 3, kb = (x >> 6) & 1, nb = x >> 7;
    if (c0 + nb * 16 >= p.C || r0 + kb * 32 >= p.Kp) continue;
    const size_t blk = (size_t)(c0 / 16 + nb) * (p.Kp / 32) + r0 / 32 + kb;
    *(v4i*)(p.dst + (blk * 64 + g * 16 + j) * 16) = t.get(nb * 16 + j, kb * 4 + g);
  }
}

template <int DT>
__device__ __forceinline__ float widen16(uint32_t pair, int hi) {
  if constexpr (DT == DT_BF16) return __builtin_bit_cast(float, hi ? (pair & 0xFFFF0000u) : (pair << 16));
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)(hi ? pair >> 16 : pair));
}

// Derivative of the activation and its value, both from one evaluation.
//   relu' = [g > 0]; silu' = s (1 + g (1 - s)), s = 1 / (1 + e^-g);
//   gelu' = P(g) + g p(g), P and p the normal distribution and its density.
template <int A>
__device__ __forceinline__ void activate_grad(float g, float& value, float& slope) {
  if constexpr (A == ACT_RELU) {
    value = activate_ffn<A>(g);
    slope = g <= 0.f ? 0.f : 1.f;
  } else if constexpr (A == ACT_SILU) {
    // e = e^-|g| by way of 2^64 e, since the hardware exponential returns 0
    // for results below 2^-126; s and 1 - s without cancellation on both sides
    const float e = ldexpf(__builtin_amdgcn_exp2f(64.f - 1.44269504088896341f * fabsf(g)), -64);
    const float r = __builtin_amdgcn_rcpf(1.f + e);
    const float s = g >= 0.f ? r : e * r, t = g >= 0.f ? e * r : r;
    value = g * s;
    slope = s * (1.f + g * t);
  } else if constexpr (A == ACT_GELU) {
    float e;
    const float P = normal_cdf(g, e);
    value = g * P;
    slope = P + g * (0.39894228040143268f * e);
  } else {
    value = g;
    slope = 1.f;
  }
}

// The gated block's pointwise backward: from dh, gate and up ([M][F]),
//   dg = dh * up * act'(gate), du = dh * act(gate)
// in fp32, rounded once to the 16-bit type the matrix products read (the
// products' own results are rounded to it as well, so this adds at most as
// much error again: normwise 0.00235 against float64 in bf16 where an fp32 form has
// 0.00166, in fp16 0.000293 and 0.000207; operands in two 16-bit parts would
// double the products, which are 85% of a large call). Written as d [M][Np] (dg, du, then zeros from 2F to Np in
// each row; null if no product reads it) and dt = d^T [2F][Mp], zeros from M to
// Mp (null likewise). F % 16 == 0.
struct GateGradArgs {
  const char *dh, *gate, *up;
  char *d, *dt;
  uint32_t M, F, Mp, Np, tiles_c, blocks;   // 64 x 64 tiles per row of tiles, and in all
  int act;
};
template <int DT>
__device__ __forceinline__ void gate_grad_tile(Tile64& tg, Tile64& tu, const GateGradArgs& p, uint32_t block) {
  const uint32_t c0 = block % p.tiles_c * 64u, r0 = block / p.tiles_c * 64u;
  const int q = threadIdx.x & 7, rp = threadIdx.x >> 3;
  const uint32_t r = r0 + 2 * rp, c = c0 + 8 * q;
  v4i in[3][2], dg[2], du[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool on = c < p.F && r + h < p.M;
    const size_t off = ((size_t)(r + h) * p.F + c) * 2;
    in[0][h] = on ? *(const v4i*)(p.dh + off) : v4i{0, 0, 0, 0};
    in[1][h] = on ? *(const v4i*)(p.gate + off) : v4i{0, 0, 0, 0};
    in[2][h] = on ? *(const v4i*)(p.up + off) : v4i{0, 0, 0, 0};
  }
  with_act(p.act, [&](auto act_c) GP_INLINE {
    constexpr int A = decltype(act_c)::value;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float og[2], ou[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float dh = widen16<DT>((uint32_t)in[0][h][i], e), g = widen16<DT>((uint32_t)in[1][h][i], e),
                      u = widen16<DT>((uint32_t)in[2][h][i], e);
          float value, slope;
          activate_grad<A>(g, value, slope);
          og[e] = dh * u * slope;
          ou[e] = dh * value;
        }
        if constexpr (DT == DT_F16) {
          dg[h][i] = (int)pack_f16x2(og[0], og[1]);
          du[h][i] = (int)pack_f16x2(ou[0], ou[1]);
        } else {
          dg[h][i] = (int)pack_bf16x2(og[0], og[1]);
          du[h][i] = (int)pack_bf16x2(ou[0], ou[1]);
        }
      }
  });
  if (p.d && c < p.F)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (r + h < p.M) {
        char* o = p.d + ((size_t)(r + h) * p.Np + c) * 2;
        *(v4i*)o = dg[h];
        *(v4i*)(o + (size_t)p.F * 2) = du[h];
      }
  if (p.d && c0 + 64 >= p.F) {
    // the last column tile fills the padding of its rows, 8 columns at a time
    const uint32_t pad = (p.Np - 2 * p.F) / 8, rows = r0 < p.M ? min(64u, p.M - r0) : 0u;
    for (uint32_t x = threadIdx.x; x < rows * pad; x += 256)
      *(v4i*)(p.d + ((size_t)(r0 + x / pad) * p.Np + 2 * p.F + x % pad * 8) * 2) = v4i{0, 0, 0, 0};
  }
  if (!p.dt) return;
  tg.put(q, rp, dg[0], dg[1]);
  tu.put(q, rp, du[0], du[1]);
  __syncthreads();
  store_transposed(tg, p.dt, c0, r0, p.F, p.Mp);
  store_transposed(tu, p.dt + (size_t)p.F * p.Mp * 2, c0, r0, p.F, p.Mp);
}

// Everything the backward products need beforehand, in one launch (a launch costs
// the host as much as a small pass takes): the pointwise backward, up to three
// copies, and the arrival counters of K splits set to zero.
struct PrepArgs {
  GateGradArgs gate;   // blocks 0: none
  CopyJob copy[3];     // blocks 0: none
  uint32_t* cnt;       // null: none
  uint32_t ncnt;
};
template <int DT>
__global__ __launch_bounds__(256) void prep_kernel(PrepArgs p) {
  __shared__ __attribute__((aligned(16))) Tile64 t0, t1;
  if (p.cnt)
    for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < p.ncnt; i += gridDim.x * 256u) p.cnt[i] = 0u;
  uint32_t b = blockIdx.x;
  if (b < p.gate.blocks) {
    gate_grad_tile<DT>(t0, t1, p.gate, b);
    return;
  }
  b -= p.gate.blocks;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (b < p.copy[i].blocks) {
      copy_tile(t0, p.copy[i], b);
      return;
    }
    b -= p.copy[i].blocks;
  }
}

}  // namespace gp
