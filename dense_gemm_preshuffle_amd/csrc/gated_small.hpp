// Small-M gated product (memory-bound regime) for gfx950:
//   h[m][f] = act(g[m][f]) * u[m][f],  g = x Wg^T, u = x Wu^T,
// for a few 16-row blocks, bound by streaming the 2F x H weights from HBM.
//
// B is the preshuffled gated layout: 16-column blocks alternate between gate
// and up rows, so the P pairs of blocks a workgroup owns give it whole output
// columns. Its WAVES waves split K in 64-byte blocks (in shares that differ by
// at most one block, so that any K does), every wave keeps two chunks of S
// blocks in flight, and the partial sums meet in LDS in wave order (the result
// is the same on every run). Wave q < MB * P then joins gate and up of output
// block q and stores it. A chunk that runs past the wave's share loads zeros
// (an offset outside the buffer resource), which add nothing.
#pragma once

#include "gp_common.hpp"

namespace gp {

struct GatedArgs {
  const char* a;      // [M][Kb] activations
  const char* b;      // preshuffled, gate and up blocks alternating
  char* c;            // [M][F]
  char* gate;         // [M][F] products to keep, or null
  char* up;
  uint32_t M, F, Kb;  // Kb = bytes per row of K
  int act;            // Act
};

template <int DT, int MB, int P, int WAVES, int S>
__global__ __launch_bounds__(WAVES * 64) void gated_small_kernel(GatedArgs p) {
  constexpr int NB = 2 * P;          // 16-column blocks of B per workgroup
  constexpr int NQ = MB * NB;        // 16 x 16 partial blocks per wave
  static_assert(MB * P <= WAVES, "one output block per wave in the epilogue");
  static_assert(WAVES * NQ * 1024 <= 160 * 1024, "LDS budget");
  __shared__ __attribute__((aligned(16))) v4f red[WAVES * NQ * 64];

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, lane_lo = lane & 15, lane_hi = lane >> 4;
  const uint32_t Kb = p.Kb;
  // each XCD takes a contiguous run of column blocks (whole lines of h per L2)
  const uint32_t pairs = p.F / 16, cols = (pairs + P - 1) / P;
  uint32_t bx = blockIdx.x % cols;
  if (cols % 8u == 0) bx = (bx % 8u) * (cols / 8u) + bx / 8u;
  const uint32_t pair0 = bx * P;
  const uint32_t npair = min((uint32_t)P, pairs - pair0);   // real pairs of this workgroup
  const uint32_t m0 = blockIdx.x / cols * (16 * MB);
  const uint32_t mrows = min(16u * MB, p.M - m0);
  const uint32_t nblk = Kb / 64;
  const uint32_t kb0 = (uint32_t)wave * nblk / WAVES, kb1 = (uint32_t)(wave + 1) * nblk / WAVES;
  const int chunks = (int)((kb1 - kb0 + S - 1) / S);

  // rows past M and blocks past the last pair lie outside their resources
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + (size_t)m0 * Kb, mrows * Kb);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.b + (size_t)pair0 * 32 * Kb, npair * 32 * Kb);
  const uint32_t a_off = lane_lo * Kb + lane_hi * 16;
  constexpr uint32_t kOOB = 0x80000000u;

  v4i af[2][S][MB], bf[2][S][NB];
  v4f acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = v4f{0.f, 0.f, 0.f, 0.f};

  auto load = [&](auto par_c, int ch) GP_INLINE {
    constexpr int par = decltype(par_c)::value;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const uint32_t k = kb0 + (uint32_t)ch * S + s;
      const uint32_t skip = k < kb1 ? 0u : kOOB;   // uniform
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        bf[par][s][nb] = buf_load16_nt(rb, (nb * 16 * Kb + k * 1024 + lane * 16) | skip, 0);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) af[par][s][mb] = buf_load16(ra, (a_off + mb * 16 * Kb + k * 64) | skip, 0);
    }
  };
  auto compute = [&](auto par_c) GP_INLINE {
    constexpr int par = decltype(par_c)::value;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) acc[mb][nb] = mfma<DT>(&bf[par][s][nb], &af[par][s][mb], acc[mb][nb]);
  };
  using P0 = std::integral_constant<int, 0>;
  using P1 = std::integral_constant<int, 1>;
  load(P0{}, 0);
  int ch = 0;
  for (; ch + 2 <= chunks; ch += 2) {
    load(P1{}, ch + 1);
    compute(P0{});
    if (ch + 2 < chunks) load(P0{}, ch + 2);
    compute(P1{});
  }
  if (ch < chunks) compute(P0{});

#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) red[(wave * NQ + mb * NB + nb) * 64 + lane] = acc[mb][nb];
  __syncthreads();
  if (wave >= MB * P) return;
  // this wave's output block: rows mb * 16 + lane_lo, columns pr * 16 + 4 * lane_hi + 0..3
  const uint32_t mb = (uint32_t)wave / P, pr = (uint32_t)wave % P;
  if (pr >= npair) return;
  v4f g = red[(mb * NB + 2 * pr) * 64 + lane], u = red[(mb * NB + 2 * pr + 1) * 64 + lane];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) {
    g += red[(w * NQ + mb * NB + 2 * pr) * 64 + lane];
    u += red[(w * NQ + mb * NB + 2 * pr + 1) * 64 + lane];
  }
  const uint32_t row = mb * 16 + lane_lo;
  if (row >= mrows) return;
  const size_t off = ((size_t)(m0 + row) * p.F + (pair0 + pr) * 16 + 4 * lane_hi) * 2;
  v4f h;
  with_act(p.act, [&](auto act_c) GP_INLINE {
    constexpr int A = decltype(act_c)::value;
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = activate<A>(g[r]) * u[r];
  });
  *(v2i*)(p.c + off) = pack_out4<DT>(h);
  if (p.gate) {
    *(v2i*)(p.gate + off) = pack_out4<DT>(g);
    *(v2i*)(p.up + off) = pack_out4<DT>(u);
  }
}

}  // namespace gp
