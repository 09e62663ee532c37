// Small-M feed-forward products (memory-bound regime) for gfx950, for a few 16-row
// blocks, bound by streaming the weights from HBM:
//   gated   h[m][f] = act(g[m][f]) * u[m][f],  g = x Wg^T, u = x Wu^T
//   linear  y[m][n] = act(z[m][n]) + res[m][n],  z = x W^T + bias
//
// B is the preshuffled layout, a workgroup owns NB of its 16-column blocks (gated:
// they alternate between gate and up rows, so that NB / 2 pairs are whole output
// columns). Its WAVES waves split K in chunks of 64 elements (in shares that
// differ by at most one, so that any K does), every wave keeps two groups of S
// chunks in flight, and the partial sums meet in LDS in wave order (the result
// is the same on every run), where a wave per output block joins gate and up, or
// adds bias and residual, and stores it. x comes row by row, 128 contiguous bytes for 8 lanes,
// and passes through a piece of LDS of the wave's own (no barrier) to the MFMA's
// layout: read from memory in that layout each lane touches another line. What
// lies past K or the wave's share is loaded as zeros (an offset outside the
// buffer resource), which add nothing. Linear, measured: one row, 4096 x 4096, 6.7 us a call
// (33.6 MB, 5.0 TB/s); 37 rows, 4096 x 14336, 27.4 (119 MB at the least, 4.3 TB/s; 132 cross the
// L2 fabric: x into every XCD's L2, and the sums of four K ranges out and back).
#pragma once

#include "gp_common.hpp"

namespace gp {

struct GatedArgs {
  const char* a;      // [M][Ka] activations
  const char* b;      // preshuffled, gate and up blocks alternating
  char* c;            // [M][F]
  char* gate;         // [M][F] products to keep, or null (linear: z)
  char* up;
  const float* bias;  // linear: fp32 [F], or null
  const char* res;    // linear: [M][F], or null
  uint32_t M, F;
  uint32_t Ka, Kb;    // bytes of K per row of x, and of the weights (whole 128-byte chunks, zeros past Ka)
  int act;            // Act
  // K split across workgroups (few column blocks, long K): ksplit workgroups share
  // a tile, the last to arrive adds their sums in order and stores it
  uint32_t ksplit;    // 1: no split
  char* part;         // [tiles][ksplit][row blocks * NB][64] v4f
  uint32_t* cnt;      // [tiles] arrival counters: zero before and after
};

// XL: 16-byte loads of x per lane and chunk: 8 XL rows; 0: a single row.
template <int DT, int XL, int NB, int WAVES, int S, bool GATED>
__global__ __launch_bounds__(WAVES * 64) void ffn_small_kernel(GatedArgs p) {
  constexpr bool ONE = XL == 0;
  constexpr int ROWS = ONE ? 1 : 8 * XL;
  constexpr int MB = (ROWS + 15) / 16;
  static_assert(!GATED || NB % 2 == 0, "whole pairs");
  constexpr int OB = GATED ? NB / 2 : NB;   // 16-column blocks of the output
  constexpr int NQ = MB * NB;        // 16 x 16 partial blocks per wave
  constexpr int XW = (ONE ? 2 : ROWS) * 128;   // LDS bytes of a wave's x (ONE: the idle lanes write past the row)
  constexpr int LDS = WAVES * (XW > NQ * 1024 ? XW : NQ * 1024);
  static_assert(LDS <= 160 * 1024, "LDS budget");
  __shared__ __attribute__((aligned(16))) char lds[LDS];

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, lane_lo = lane & 15, lane_hi = lane >> 4;
  const uint32_t Ka = p.Ka, Kb = p.Kb;
  // each XCD takes a contiguous run of column blocks (whole lines of h per L2)
  const uint32_t blocks = p.F / 16, cols = (blocks + OB - 1) / OB;
  const uint32_t tiles = gridDim.x / p.ksplit, tile = blockIdx.x % tiles, kz = blockIdx.x / tiles;
  uint32_t bx = tile % cols;
  if (cols % 8u == 0) bx = (bx % 8u) * (cols / 8u) + bx / 8u;
  const uint32_t block0 = bx * OB;
  const uint32_t nblock = min((uint32_t)OB, blocks - block0);   // real blocks of this workgroup
  const uint32_t m0 = tile / cols * ROWS;
  const uint32_t mrows = min((uint32_t)ROWS, p.M - m0);
  const uint32_t nchunk = Kb / 128;
  const uint32_t share = kz * WAVES + wave, shares = p.ksplit * WAVES;   // of K's chunks
  const uint32_t kc0 = share * nchunk / shares, kc1 = (share + 1) * nchunk / shares;
  const int groups = (int)((kc1 - kc0 + S - 1) / S);

  // rows past M and blocks past the last lie outside their resources
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + (size_t)m0 * Ka, mrows * Ka);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.b + (size_t)block0 * (NB / OB * 16) * Kb, nblock * (NB / OB * 16) * Kb);
  constexpr uint32_t kOOB = 0x80000000u;
  // x load i of a lane: 16-byte piece lane % 8 of row 8 i + lane / 8. Piece c of
  // row m stands in LDS at c ^ (m / 2 % 8): the 16 rows of one piece, which an
  // MFMA operand reads together, lie in different banks.
  char* xw = lds + wave * XW;
  const uint32_t xcol = ONE ? 4 * lane : 16 * (lane & 7);
  const uint32_t x_off = ONE ? (lane < 32 ? xcol : kOOB) : (lane >> 3) * Ka + xcol;

  v4i xr[2][S][XL > 0 ? XL : 1], bf[2][S][2][NB];
  v4f acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = v4f{0.f, 0.f, 0.f, 0.f};

  // the chunk's offset is scalar; bounds are checked on the lane's part alone
  auto load = [&](auto par_c, int gr) GP_INLINE {
    constexpr int par = decltype(par_c)::value;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const uint32_t k = kc0 + (uint32_t)gr * S + s;
      const uint32_t skip = S == 1 || k < kc1 ? 0u : kOOB;   // uniform
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        bf[par][s][0][nb] = buf_load16_nt(rb, (nb * 16 * Kb + lane * 16) | skip, k * 2048);
        bf[par][s][1][nb] = buf_load16_nt(rb, (nb * 16 * Kb + lane * 16 + 1024) | skip, k * 2048);
      }
      // (or-ed in: a sum would pass 2^32 for the longest rows)
      const uint32_t past = (128 * k + xcol < Ka ? 0u : kOOB) | skip;
      if constexpr (ONE) xr[par][s][0][0] = buf_load4(ra, x_off | past, 128 * k);
#pragma unroll
      for (int i = 0; i < XL; ++i) xr[par][s][i] = buf_load16(ra, (x_off + 8 * i * Ka) | past, 128 * k);
    }
  };
  auto compute = [&](auto par_c) GP_INLINE {
    constexpr int par = decltype(par_c)::value;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if constexpr (ONE) *(int*)(xw + 4 * lane) = xr[par][s][0][0];
#pragma unroll
      for (int i = 0; i < XL; ++i) {
        const int m = 8 * i + (lane >> 3);
        *(v4i*)(xw + m * 128 + (((lane & 7) ^ ((m >> 1) & 7)) * 16)) = xr[par][s][i];
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const int m = ONE ? 0 : (mb * 16 + lane_lo) % ROWS;   // rows past ROWS repeat and are not stored
          const v4i xf = *(const v4i*)(xw + m * 128 + (((4 * t + lane_hi) ^ ((m >> 1) & 7)) * 16));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = mfma<DT>(&bf[par][s][t][nb], &xf, acc[mb][nb]);
        }
    }
  };
  using P0 = std::integral_constant<int, 0>;
  using P1 = std::integral_constant<int, 1>;
  if (groups > 0) {
    load(P0{}, 0);
    int gr = 0;
    for (; gr + 2 <= groups; gr += 2) {
      load(P1{}, gr + 1);
      compute(P0{});
      if (gr + 2 < groups) load(P0{}, gr + 2);
      compute(P1{});
    }
    if (gr < groups) compute(P0{});
  }

  __syncthreads();   // the sums take the place of the waves' x
  v4f* red = (v4f*)lds;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) red[(wave * NQ + mb * NB + nb) * 64 + lane] = acc[mb][nb];
  __syncthreads();
  // an output block per wave and turn: rows mb * 16 + lane_lo, columns
  // ob * 16 + 4 * lane_hi + 0..3
  constexpr int NV = NB / OB;   // sums of an output
  auto sum_waves = [&](uint32_t q, v4f (&v)[NV]) GP_INLINE {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = red[(NV * q + i) * 64 + lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) v[i] += red[(w * NQ + NV * q + i) * 64 + lane];
    }
  };
  constexpr uint32_t QB = NV * 1024, PB = MB * OB * QB;   // bytes of an output block's sums, and of a workgroup's
  const __amdgpu_buffer_rsrc_t rp = make_rsrc(p.part + (size_t)tile * p.ksplit * PB, p.ksplit > 1 ? p.ksplit * PB : 0);
  if (p.ksplit > 1) {
    for (uint32_t q = (uint32_t)wave; q < MB * OB; q += WAVES) {
      v4f v[NV];
      sum_waves(q, v);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        buf_store16_coh(__builtin_bit_cast(v4i, v[i]), rp, kz * PB + q * QB + i * 1024 + lane * 16);
    }
    // (the word is written after a barrier: the sums in LDS are done with)
    if (!last_to_arrive(p.cnt + tile, p.ksplit, (volatile uint32_t*)lds)) return;
  }
  for (uint32_t q = (uint32_t)wave; q < MB * OB; q += WAVES) {
    const uint32_t mb = q / OB, ob = q % OB, row = mb * 16 + lane_lo;
    if (ob >= nblock || row >= mrows) continue;
    v4f v[NV];
    if (p.ksplit > 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = v4f{0.f, 0.f, 0.f, 0.f};
      for (uint32_t z = 0; z < p.ksplit; ++z)
#pragma unroll
        for (int i = 0; i < NV; ++i)
          v[i] += __builtin_bit_cast(v4f, buf_load16_coh(rp, z * PB + q * QB + i * 1024 + lane * 16));
    } else {
      sum_waves(q, v);
    }
    const uint32_t col = (block0 + ob) * 16 + 4 * lane_hi;
    const size_t off = ((size_t)(m0 + row) * p.F + col) * 2;
    if constexpr (GATED) {
      v4f h;
      with_act(p.act, [&](auto act_c) GP_INLINE {
        constexpr int A = decltype(act_c)::value;
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = activate_ffn<A>(v[0][r]) * v[1][r];
      });
      *(v2i*)(p.c + off) = pack_out4<DT>(h);
      if (p.gate) {
        *(v2i*)(p.gate + off) = pack_out4<DT>(v[0]);
        *(v2i*)(p.up + off) = pack_out4<DT>(v[1]);
      }
    } else {
      if (p.bias) v[0] += *(const v4f*)(p.bias + col);
      if (p.gate) *(v2i*)(p.gate + off) = pack_out4<DT>(v[0]);
      with_act(p.act, [&](auto act_c) GP_INLINE {
        constexpr int A = decltype(act_c)::value;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[0][r] = activate_ffn<A>(v[0][r]);
      });
      if (p.res) v[0] += widen4<DT>(*(const v2i*)(p.res + off));
      *(v2i*)(p.c + off) = pack_out4<DT>(v[0]);
    }
  }
}

}  // namespace gp
