// Products with 4-bit weights and group scales for few rows, on gfx950:
//   y[m][n] = sum_k x[m][k] s[n][k / G] (q[n][k] - z[n][k / G]),
// x in BF16 or FP16, q a 4-bit integer; also the gated form
// act(x Wg^T) * (x Wu^T) on two such weights. Bound by streaming the 4-bit
// weights from HBM.
//
// The integers are multiplied on the 16 x 16 x 32 MFMA of x's type: every
// q - z (and q + 8) is a whole number below 256 and exact in both types. A
// group's products are accumulated apart, in fp32, and joined to the row's sum
// with the group's scale, so that no weight is ever rounded:
//   y += s * sum_group x (q - z).
// A nibble u = q + 8 in 0 .. 15, read as an FP8 E4M3 code, is the number
// u * 2^-9 (codes below 8 are the subnormals, 8 .. 15 the first binade), so one
// conversion instruction with the scale 2^9 makes two operands.
//   FP16: u is converted and 8 + z subtracted, exactly, on packed halves.
//   BF16 has no packed subtract: the MFMA takes u itself, and the group's sum
//     of x times (8 + z) is subtracted in fp32 before the scale. The sum of x
//     comes from one more MFMA against ones, whose result stands in the lanes
//     that need it and which serves every column block. The subtraction
//     loses at most a few fp32 steps of a sum of at most 16 |x| per element,
//     far below the output's rounding. Where x holds infinities (or the sums
//     overflow) it gives NaN; such outputs are computed again, one by one, from
//     the formula.
//
// Layout: 16 output columns x 128 K per block of 1 KiB. Lane l of a wave reads
// its 16 bytes at 16 l: column l % 16, K piece l / 16; dword j holds the eight
// elements of K step j, k = 32 j + 8 (l / 16) + i, element i < 4 in the low
// nibble of byte i, the others in the high nibbles. Scales and zero points
// follow, per column block and 128 K (or per longer group), as [16 columns]
// [groups inside the block], so that a lane's are one load.
//
// A workgroup owns NB column blocks and up to 16 MB rows; its waves split K in
// whole blocks, each with two chunks of S blocks in flight, and their sums meet
// in LDS in wave order (the same bits on every run).
#pragma once

#include "gp_common.hpp"

namespace gp {

struct W4Args {
  const char* x;       // [M][K]
  const char* w;       // laid-out weights
  const char* s;       // laid-out scales (x's type)
  const char* z;       // laid-out zero points (int8) or null
  const float* bias;   // fp32 [N] or null
  char* y;             // [M][N]
  uint32_t M, N, K;    // N: columns of y (gated: F)
  uint32_t nblk;       // 16-column blocks of the weights
  uint32_t sshift;     // log2 of 128-element blocks per scale (0: one or several scales per block)
  int act;             // Act
  int gated;           // gate and up blocks alternate
};

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// Eight nibbles -> eight 16-bit operands. BF16: u = q + 8. FP16: u + off
// (off = -(8 + z) in both halves).
template <int DT>
__device__ __forceinline__ v4i unpack_w4(int d, v2h off) {
  const int lo = d & 0x0F0F0F0F, hi = (int)((uint32_t)d >> 4) & 0x0F0F0F0F;
  v4i o;
  if constexpr (DT == DT_BF16) {
    o[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, false));
    o[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, true));
    o[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, false));
    o[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, true));
  } else {
    const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.f, false);
    const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.f, true);
    const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.f, false);
    const v2h e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.f, true);
    o[0] = __builtin_bit_cast(int, (v2h)(a + off));
    o[1] = __builtin_bit_cast(int, (v2h)(b + off));
    o[2] = __builtin_bit_cast(int, (v2h)(c + off));
    o[3] = __builtin_bit_cast(int, (v2h)(e + off));
  }
  return o;
}

template <int DT>
__device__ __forceinline__ float half_to_float(uint32_t bits) {
  if constexpr (DT == DT_BF16) return __builtin_bit_cast(float, bits << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

// One output from the formula, for the sums that the split of q - z into u and
// 8 + z cannot give (see above).
template <int DT, int SG>
__device__ __forceinline__ float w4_direct(const W4Args& p, uint32_t m, uint32_t nb, uint32_t col) {
  const uint32_t kblk = (p.K + 127) / 128, sblk = (kblk + (1u << p.sshift) - 1) >> p.sshift;
  const uint16_t* xr = (const uint16_t*)(p.x + (size_t)m * p.K * 2);
  float sum = 0.f;
  for (uint32_t k = 0; k < p.K; ++k) {
    const uint32_t b = k / 128, j = k / 32 % 4, hi = k / 8 % 4, i = k % 8;
    const uint32_t byte = (uint8_t)p.w[((size_t)nb * kblk + b) * 1024 + (hi * 16 + col) * 16 + j * 4 + (i & 3)];
    const int u = (int)(i < 4 ? byte & 15u : byte >> 4);
    const size_t g = (((size_t)nb * sblk + (b >> p.sshift)) * 16 + col) * SG + (SG > 1 ? j * SG / 4 : 0);
    const int z = p.z ? (int)(int8_t)p.z[g] : 0;
    const float s = half_to_float<DT>(((const uint16_t*)p.s)[g]);
    sum = fmaf(half_to_float<DT>(xr[k]), s * (float)(u - 8 - z), sum);
  }
  return sum;
}

// ONE: a single row (M = 1): only the first result register of a block counts.
template <int DT, int MB, int NB, int WAVES, int S, int SG, bool ZERO, bool ONE>
__global__ __launch_bounds__(WAVES * 64) void w4a16_kernel(W4Args p) {
  constexpr int NQ = MB * NB;
  constexpr int R = ONE ? 1 : 4;
  constexpr int STEPS = 4 / SG;         // K steps of 32 per scale inside a block
  static_assert(!ONE || MB == 1, "one row");
  static_assert(WAVES * NQ * 64 * R * 4 <= 160 * 1024, "LDS budget");
  __shared__ __attribute__((aligned(16))) float red[WAVES * NQ * 64 * R];

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, lane_lo = lane & 15, lane_hi = lane >> 4;
  const uint32_t K = p.K, Kb = 2 * K;
  const uint32_t kblk = (K + 127) / 128, sblk = (kblk + (1u << p.sshift) - 1) >> p.sshift;
  const uint32_t cols = (p.nblk + NB - 1) / NB;
  uint32_t bx = blockIdx.x % cols;
  if (cols % 8u == 0) bx = (bx % 8u) * (cols / 8u) + bx / 8u;   // a contiguous run of columns per XCD
  const uint32_t nb0 = bx * NB;
  const uint32_t nreal = min((uint32_t)NB, p.nblk - nb0);
  const uint32_t m0 = blockIdx.x / cols * (16 * MB);
  const uint32_t mrows = min(16u * MB, p.M - m0);
  const uint32_t kb0 = (uint32_t)((uint64_t)wave * kblk / WAVES), kb1 = (uint32_t)((uint64_t)(wave + 1) * kblk / WAVES);
  const int chunks = (int)((kb1 - kb0 + S - 1) / S);

  constexpr uint32_t kOOB = 0x80000000u;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x + (size_t)m0 * Kb, mrows * Kb);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w + (size_t)nb0 * kblk * 1024, nreal * kblk * 1024);
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(p.s + (size_t)nb0 * sblk * (32 * SG), nreal * sblk * (32 * SG));
  const __amdgpu_buffer_rsrc_t rz =
      make_rsrc(ZERO ? p.z + (size_t)nb0 * sblk * (16 * SG) : nullptr, ZERO ? nreal * sblk * (16 * SG) : 0);
  // rows past the last read it again (their results are not stored)
  uint32_t x_off[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) x_off[mb] = min((uint32_t)(mb * 16 + lane_lo), mrows - 1) * Kb + lane_hi * 16;

  v4i xf[2][S][4][MB], wf[2][S][NB];
  uint32_t sf[2][S][NB][SG == 4 ? 2 : 1], zf[2][S][NB];
  v4f acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = v4f{0.f, 0.f, 0.f, 0.f};

  auto load = [&](auto par_c, int ch) GP_INLINE {
    constexpr int par = decltype(par_c)::value;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const uint32_t b = kb0 + (uint32_t)ch * S + s;
      const uint32_t skip = b < kb1 ? 0u : kOOB;   // uniform: past the wave's share
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        wf[par][s][nb] = buf_load16_nt(rw, ((nb * kblk + b) * 1024 + lane * 16) | skip, 0);
        const uint32_t g = ((nb * sblk + (b >> p.sshift)) * 16 + lane_lo) * SG;
        if constexpr (SG == 1) sf[par][s][nb][0] = __builtin_amdgcn_raw_buffer_load_b16(rs, (g * 2) | skip, 0, 0);
        else if constexpr (SG == 2) sf[par][s][nb][0] = buf_load4(rs, (g * 2) | skip, 0);
        else {
          const v2i t = buf_load8(rs, (g * 2) | skip, 0);
          sf[par][s][nb][0] = (uint32_t)t[0];
          sf[par][s][nb][1] = (uint32_t)t[1];
        }
        if constexpr (ZERO) {
          if constexpr (SG == 1) zf[par][s][nb] = __builtin_amdgcn_raw_buffer_load_b8(rz, g | skip, 0, 0);
          else if constexpr (SG == 2) zf[par][s][nb] = __builtin_amdgcn_raw_buffer_load_b16(rz, g | skip, 0, 0);
          else zf[par][s][nb] = buf_load4(rz, g | skip, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // K is whole steps of 32, not whole blocks
        const uint32_t off = 256 * b + 64 * j, xskip = (b < kb1 && off < Kb) ? 0u : kOOB;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) xf[par][s][j][mb] = buf_load16(rx, (x_off[mb] + off) | xskip, 0);
      }
    }
  };
  const v4i ones = v4i{0x3F803F80, 0x3F803F80, 0x3F803F80, 0x3F803F80};
  auto compute = [&](auto par_c) GP_INLINE {
    constexpr int par = decltype(par_c)::value;
    static_for<0, S>([&](auto s_c) GP_INLINE {
      constexpr int s = decltype(s_c)::value;
      static_for<0, SG>([&](auto g_c) GP_INLINE {
        constexpr int g = decltype(g_c)::value;
        v4f sum[MB];
        if constexpr (DT == DT_BF16)
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            sum[mb] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = g * STEPS; j < (g + 1) * STEPS; ++j) sum[mb] = mfma<DT>(&xf[par][s][j][mb], &ones, sum[mb]);
          }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const uint32_t sw = sf[par][s][nb][g / 2];
          const float sc = half_to_float<DT>(SG == 1 ? sw : (g % 2 ? sw >> 16 : sw & 0xFFFFu));
          const int off = ZERO ? 8 + (int)(int8_t)(zf[par][s][nb] >> (8 * g)) : 8;
          v2h hoff;
          if constexpr (DT == DT_F16) hoff[0] = hoff[1] = (_Float16)(-off);
          v4f part[MB];
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) part[mb] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = g * STEPS; j < (g + 1) * STEPS; ++j) {
            const v4i wv = unpack_w4<DT>(wf[par][s][nb][j], hoff);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) part[mb] = mfma<DT>(&xf[par][s][j][mb], &wv, part[mb]);
          }
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int r = 0; r < R; ++r) {
              float t = part[mb][r];
              if constexpr (DT == DT_BF16) t = fmaf(-(float)off, sum[mb][r], t);
              acc[mb][nb][r] = fmaf(sc, t, acc[mb][nb][r]);
            }
        }
      });
    });
  };
  using P0 = std::integral_constant<int, 0>;
  using P1 = std::integral_constant<int, 1>;
  if (chunks > 0) {
    load(P0{}, 0);
    int ch = 0;
    for (; ch + 2 <= chunks; ch += 2) {
      load(P1{}, ch + 1);
      compute(P0{});
      if (ch + 2 < chunks) load(P0{}, ch + 2);
      compute(P1{});
    }
    if (ch < chunks) compute(P0{});
  }

#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < R; ++r) red[((wave * NQ + mb * NB + nb) * R + r) * 64 + lane] = acc[mb][nb][r];
  __syncthreads();

  // output blocks of the workgroup: row block mb, column block(s) c
  const int per = p.gated ? NB / 2 : NB;
  for (int q = wave; q < MB * per; q += WAVES) {
    const int mb = q / per, c = q % per, b0 = p.gated ? 2 * c : c;
    const uint32_t nb = nb0 + b0;
    if (nb >= p.nblk) continue;
    auto total = [&](int blk, float* v) GP_INLINE {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) t += red[((w * NQ + mb * NB + blk) * R + r) * 64 + lane];
        v[r] = t;
      }
    };
    float v[R], u[R];
    total(b0, v);
    if (p.gated) total(b0 + 1, u);
    const uint32_t n = (p.gated ? nb / 2 : nb) * 16 + lane_lo;
    if (n >= p.N) continue;
    const float bias = p.bias ? p.bias[n] : 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t row = mb * 16 + 4 * lane_hi + r;
      if (row >= mrows) continue;
      if constexpr (DT == DT_BF16) {
        if (v[r] != v[r]) v[r] = w4_direct<DT, SG>(p, m0 + row, nb, lane_lo);
        if (p.gated && u[r] != u[r]) u[r] = w4_direct<DT, SG>(p, m0 + row, nb + 1, lane_lo);
      }
      float o = 0.f;
      with_act(p.act, [&](auto act_c) GP_INLINE { o = activate<decltype(act_c)::value>(v[r] + bias); });
      if (p.gated) o *= u[r];
      const uint32_t two = DT == DT_F16 ? pack_f16x2(o, 0.f) : pack_bf16x2(o, 0.f);
      *(uint16_t*)(p.y + ((size_t)(m0 + row) * p.N + n) * 2) = (uint16_t)two;
    }
  }
}

}  // namespace gp
