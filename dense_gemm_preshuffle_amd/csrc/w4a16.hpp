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
// conversion instruction with the scale 2^9 makes two operands: 7 instructions
// for 8 weights, which matters since the vector unit has about 80 instruction
// slots per KiB of weights at the full HBM rate. The 8 is taken off by the matrix
// instructions: a group's accumulator starts from sum x (-8), a product with a
// constant operand whose result serves every column block; a zero point adds
// z/8 of the same sum. What cancels there is at most 23 |x| per element
// (16 |x| + |z| |x| with zero points) in fp32, far below the output's rounding.
// Where x or a scale is not finite, or the sums overflow, no finite number comes
// out of that; a wave that holds such a sum goes over its share of K again, with
// q - z itself as the operand (a whole number of at most 135, exact in both
// types), and replaces the sums that were not finite alone.
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
// in LDS in wave order (the same bits on every run). x comes row by row, 256
// contiguous bytes for 16 lanes, and passes through a piece of LDS of the
// wave's own (no barrier) to the MFMA's layout: read from memory in that layout
// each of the 64 lanes touches another line of x, and the rows' loads took as
// long as the weights' (16 x 4091 x 7168: 10.3 us).
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
  // K split across workgroups (few column blocks, long K): ksplit workgroups share
  // a tile, the last to arrive adds their sums in order and stores it
  uint32_t ksplit;     // 1: no split
  char* part;          // [tiles][ksplit][row blocks * NB][result registers][64] fp32
  uint32_t* cnt;       // [tiles] arrival counters: zero before and after
};

// Eight nibbles u = q + 8 -> eight 16-bit operands.
template <int DT>
__device__ __forceinline__ v4i unpack_w4(int d) {
  const int lo = d & 0x0F0F0F0F, hi = (int)((uint32_t)d >> 4) & 0x0F0F0F0F;
  v4i o;
  if constexpr (DT == DT_BF16) {
    o[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, false));
    o[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, true));
    o[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, false));
    o[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, true));
  } else {
    o[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.f, false));
    o[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.f, true));
    o[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.f, false));
    o[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.f, true));
  }
  return o;
}

template <int DT>
__device__ __forceinline__ float half_to_float(uint32_t bits) {
  if constexpr (DT == DT_BF16) return __builtin_bit_cast(float, bits << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

// Eight nibbles u = q + 8 -> eight 16-bit operands (u - 8 - z) f, without the
// conversion's split: for the sums that it cannot give (see above).
template <int DT>
__device__ __forceinline__ v4i unpack_w4_less(int d, int z, float f) {
  v4i o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t at = i < 2 ? 16 * i : 16 * (i - 2) + 4;   // elements 2 i, 2 i + 1
    const float lo = f * (float)((int)((uint32_t)d >> at & 15u) - 8 - z),
                hi = f * (float)((int)((uint32_t)d >> (at + 8) & 15u) - 8 - z);
    o[i] = (int)(DT == DT_F16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi));
  }
  return o;
}

// XL: 16-byte loads of x per lane and block: 1, 4, 8 or 16 serve 4, 16, 32 or
// 64 rows; 0: a single row, one dword per lane.
template <int DT, int XL, int NB, int WAVES, int S, int SG, bool ZERO>
__global__ __launch_bounds__(WAVES * 64) void w4a16_kernel(W4Args p) {
  constexpr bool ONE = XL == 0;
  constexpr int ROWS = ONE ? 1 : 4 * XL;
  constexpr int MB = (ROWS + 15) / 16;
  constexpr int NQ = MB * NB;
  constexpr int R = ONE ? 1 : 4;        // result registers that hold rows
  constexpr int STEPS = 4 / SG;         // K steps of 32 per scale inside a block
  constexpr float kMaxFloat = 3.402823466e38f;
  static_assert(WAVES * (ROWS * 256 + NQ * 64 * R * 4) <= 160 * 1024, "LDS budget");
  __shared__ __attribute__((aligned(16))) char xs[WAVES * ROWS * 256];
  __shared__ __attribute__((aligned(16))) float red[WAVES * NQ * 64 * R];

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, lane_lo = lane & 15, lane_hi = lane >> 4;
  const uint32_t K = p.K, Kb = 2 * K;
  const uint32_t kblk = (K + 127) / 128, sblk = (kblk + (1u << p.sshift) - 1) >> p.sshift;
  const uint32_t cols = (p.nblk + NB - 1) / NB;
  const uint32_t tiles = gridDim.x / p.ksplit, tile = blockIdx.x % tiles, kz = blockIdx.x / tiles;
  uint32_t bx = tile % cols;
  if (cols % 8u == 0) bx = (bx % 8u) * (cols / 8u) + bx / 8u;   // a contiguous run of columns per XCD
  const uint32_t nb0 = bx * NB;
  const uint32_t nreal = min((uint32_t)NB, p.nblk - nb0);
  const uint32_t m0 = tile / cols * ROWS;
  const uint32_t mrows = min((uint32_t)ROWS, p.M - m0);
  const uint32_t share = kz * WAVES + wave, shares = p.ksplit * WAVES;   // of K's blocks
  const uint32_t kb0 = share * kblk / shares, kb1 = (share + 1) * kblk / shares;
  const int chunks = (int)((kb1 - kb0 + S - 1) / S);

  // rows past M and column blocks past the last lie outside their resources
  constexpr uint32_t kOOB = 0x80000000u;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x + (size_t)m0 * Kb, mrows * Kb);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w + (size_t)nb0 * kblk * 1024, nreal * kblk * 1024);
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(p.s + (size_t)nb0 * sblk * (32 * SG), nreal * sblk * (32 * SG));
  const __amdgpu_buffer_rsrc_t rz =
      make_rsrc(ZERO ? p.z + (size_t)nb0 * sblk * (16 * SG) : nullptr, ZERO ? nreal * sblk * (16 * SG) : 0);
  // x: load i of a lane is 16-byte piece lane % 16 of row 4 i + lane / 16. In
  // LDS piece c of row m stands at c ^ (m % 16), so that the 16 rows of one
  // piece, which an MFMA operand reads together, lie in different banks.
  char* xw = xs + wave * ROWS * 256;
  const uint32_t xcol = ONE ? 4 * lane : 16 * lane_lo;
  const uint32_t x_off = (ONE ? 0 : lane_hi * Kb) + xcol;

  v4i xr[2][S][XL > 0 ? XL : 1], wf[2][S][NB];
  uint32_t sf[2][S][NB][SG == 4 ? 2 : 1], zf[2][S][NB];
  v4f acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = v4f{0.f, 0.f, 0.f, 0.f};

  // The block's offset is scalar; bounds are checked on the lane's part alone,
  // so what lies past the share of a wave (S > 1) or past K gets a lane offset
  // outside the resource.
  auto load = [&](auto par_c, int ch) GP_INLINE {
    constexpr int par = decltype(par_c)::value;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const uint32_t b = kb0 + (uint32_t)ch * S + s;
      const uint32_t skip = S == 1 || b < kb1 ? 0u : kOOB;
      const uint32_t xo = (256 * b + xcol < Kb ? x_off : kOOB) | skip;
      if constexpr (ONE) xr[par][s][0][0] = buf_load4(rx, xo, 256 * b);
#pragma unroll
      for (int i = 0; i < XL; ++i) xr[par][s][i] = buf_load16(rx, xo + 4 * i * Kb, 256 * b);
      const uint32_t g = (b >> p.sshift) * 16 * SG;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        wf[par][s][nb] = buf_load16_nt(rw, (nb * kblk * 1024 + lane * 16) | skip, b * 1024);
        const uint32_t go = (nb * sblk * 16 + lane_lo) * SG;
        if constexpr (SG == 1) sf[par][s][nb][0] = __builtin_amdgcn_raw_buffer_load_b16(rs, (go * 2) | skip, g * 2, 0);
        else if constexpr (SG == 2) sf[par][s][nb][0] = buf_load4(rs, (go * 2) | skip, g * 2);
        else {
          const v2i t = buf_load8(rs, (go * 2) | skip, g * 2);
          sf[par][s][nb][0] = (uint32_t)t[0];
          sf[par][s][nb][1] = (uint32_t)t[1];
        }
        if constexpr (ZERO) {
          if constexpr (SG == 1) zf[par][s][nb] = __builtin_amdgcn_raw_buffer_load_b8(rz, go | skip, g, 0);
          else if constexpr (SG == 2) zf[par][s][nb] = __builtin_amdgcn_raw_buffer_load_b16(rz, go | skip, g, 0);
          else zf[par][s][nb] = buf_load4(rz, go | skip, g);
        }
      }
    }
  };
  constexpr int kM8 = DT == DT_BF16 ? (int)0xC100C100 : (int)0xC800C800;
  const v4i minus8 = v4i{kM8, kM8, kM8, kM8};
  auto compute = [&](auto par_c) GP_INLINE {
    constexpr int par = decltype(par_c)::value;
    static_for<0, S>([&](auto s_c) GP_INLINE {
      constexpr int s = decltype(s_c)::value;
      if constexpr (ONE) *(int*)(xw + 4 * lane) = xr[par][s][0][0];
#pragma unroll
      for (int i = 0; i < XL; ++i) {
        const int m = 4 * i + lane_hi;
        *(v4i*)(xw + m * 256 + ((lane_lo ^ (m & 15)) * 16)) = xr[par][s][i];
      }
      int xg = 0;
      static_for<0, SG>([&](auto g_c) GP_INLINE {
        constexpr int g = decltype(g_c)::value;
        // rows past ROWS (a single row, or four) repeat; their results are not stored
        v4i xf[STEPS][MB];
#pragma unroll
        for (int j = 0; j < STEPS; ++j)
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            const int c = 4 * (g * STEPS + j) + lane_hi;
            const int m = ONE ? 0 : (mb * 16 + lane_lo) % ROWS;
            xf[j][mb] = *(const v4i*)(xw + xg + m * 256 + ((c ^ (m & 15)) * 16));
          }
        v4f sum[MB];   // -8 times the sum of x
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          sum[mb] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < STEPS; ++j) sum[mb] = mfma<DT>(&xf[j][mb], &minus8, sum[mb]);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const uint32_t sw = sf[par][s][nb][g / 2];
          const float sc = half_to_float<DT>(SG == 1 ? sw : (g % 2 ? sw >> 16 : sw & 0xFFFFu));
          const float z8 = ZERO ? 0.125f * (float)(int)(int8_t)(zf[par][s][nb] >> (8 * g)) : 0.f;
          v4f part[MB];
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) part[mb] = sum[mb];
#pragma unroll
          for (int j = 0; j < STEPS; ++j) {
            const v4i wv = unpack_w4<DT>(wf[par][s][nb][g * STEPS + j]);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) part[mb] = mfma<DT>(&xf[j][mb], &wv, part[mb]);
          }
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int r = 0; r < R; ++r)
              acc[mb][nb][r] = fmaf(sc, ZERO ? fmaf(z8, sum[mb][r], part[mb][r]) : part[mb][r], acc[mb][nb][r]);
        }
        // Left free, the compiler interleaves the groups of many rows until
        // their operands no longer fit the registers: the next group's LDS
        // address is made to depend on this group's results.
        if constexpr (MB > 1 && SG > 1)
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) asm volatile("" : "+v"(xg), "+v"(acc[mb][nb]));
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

  float probe = 0.f;   // 0 times every sum: NaN if one is not finite
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        red[((wave * NQ + mb * NB + nb) * R + r) * 64 + lane] = acc[mb][nb][r];
        probe = fmaf(acc[mb][nb][r], 0.f, probe);
      }
  // Sums that are not finite, again with q - z as the operand: an infinity of x
  // or of a scale meets the weight that the formula has there, 0 included. In BF16
  // the operands carry 2^-16, which keeps the products of finite x finite (FP16's
  // cannot overflow); a scale that is not finite goes into the operand, since a
  // product x (q - z) of 0 would hide it. One column block at a time and
  // straight from memory, whatever the number of such sums: 64 x 8192 x 28672 in
  // BF16 76 us clean, 219 with a NaN in one row, 366 with nothing but NaN; one row
  // 23, 34, 77 (output by output each would take K dependent steps).
  if (__builtin_expect(__any(!(probe == 0.f)), 0)) for (uint32_t blk = 0; blk < nreal; ++blk) {
    constexpr int kDown = DT == DT_BF16 ? 16 : 0;
    v4f sum[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) sum[mb] = v4f{0.f, 0.f, 0.f, 0.f};
    // steps of 32 K; few rows: not unrolled, for the registers of two workgroups per CU
#pragma unroll(XL <= 1 ? 1 : XL <= 8 ? 4 : 2)
    for (uint32_t step = 4 * kb0; step < 4 * kb1; ++step) {
      const uint32_t b = step / 4, j = step % 4, go = (blk * sblk * 16 + lane_lo) * SG + (SG > 1 ? j * SG / 4 : 0),
                     gs = (b >> p.sshift) * 16 * SG, col = 64 * j + 16 * lane_hi;
      const int wd = buf_load4(rw, blk * kblk * 1024 + lane * 16 + 4 * j, b * 1024);
      float sc = half_to_float<DT>(__builtin_amdgcn_raw_buffer_load_b16(rs, go * 2, gs * 2, 0));
      const int z = ZERO ? (int)(int8_t)__builtin_amdgcn_raw_buffer_load_b8(rz, go, gs, 0) : 0;
      float f = DT == DT_BF16 ? 0x1p-16f : 1.f;
      if (!(fabsf(sc) <= kMaxFloat)) {
        f = sc;
        sc = 1.f;
      }
      const v4i wv = unpack_w4_less<DT>(wd, z, f);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const uint32_t m = ONE ? 0 : (mb * 16 + lane_lo) % ROWS;
        const v4i xv = buf_load16(rx, 256 * b + col < Kb ? m * Kb + col : kOOB, 256 * b);
        const v4f part = mfma<DT>(&xv, &wv, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int r = 0; r < R; ++r) sum[mb][r] = fmaf(sc, part[r], sum[mb][r]);
      }
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float& t = red[((wave * NQ + mb * NB + blk) * R + r) * 64 + lane];
        if (!(fabsf(t) <= kMaxFloat)) t = ldexpf(sum[mb][r], kDown);
      }
  }
  __syncthreads();

  constexpr uint32_t PB = NQ * R * 256;   // bytes of one workgroup's sums
  const __amdgpu_buffer_rsrc_t rp = make_rsrc(p.part + (size_t)tile * p.ksplit * PB, p.ksplit > 1 ? p.ksplit * PB : 0);
  auto sum_waves = [&](int qr) GP_INLINE {   // block and register qr
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) t += red[(w * NQ * R + qr) * 64 + lane];
    return t;
  };
  if (p.ksplit > 1) {
    for (int qr = wave; qr < NQ * R; qr += WAVES) buf_store4_coh(sum_waves(qr), rp, kz * PB + qr * 256 + lane * 4);
    if (!last_to_arrive(p.cnt + tile, p.ksplit, (volatile uint32_t*)xs)) return;   // (x is done with)
  }
  // one wave per output block (row block mb, column block or pair c) and result
  // register r
  const int per = p.gated ? NB / 2 : NB;
  for (int q = wave; q < MB * per * R; q += WAVES) {
    const int r = q % R, c = q / R % per, mb = q / R / per, b0 = p.gated ? 2 * c : c;
    const uint32_t nb = nb0 + b0;
    const uint32_t n = (p.gated ? nb / 2 : nb) * 16 + lane_lo;
    const uint32_t row = mb * 16 + 4 * lane_hi + r;
    if (nb >= p.nblk || n >= p.N || row >= mrows) continue;
    auto total = [&](int blk) GP_INLINE {
      const int qr = (mb * NB + blk) * R + r;
      if (p.ksplit <= 1) return sum_waves(qr);
      float t = 0.f;
      for (uint32_t z = 0; z < p.ksplit; ++z) t += buf_load4_coh(rp, z * PB + qr * 256 + lane * 4);
      return t;
    };
    float o = total(b0) + (p.bias ? p.bias[n] : 0.f);
    with_act(p.act, [&](auto act_c) GP_INLINE { o = activate_ffn<decltype(act_c)::value>(o); });
    if (p.gated) o *= total(b0 + 1);
    const uint32_t two = DT == DT_F16 ? pack_f16x2(o, 0.f) : pack_bf16x2(o, 0.f);
    *(uint16_t*)(p.y + ((size_t)(m0 + row) * p.N + n) * 2) = (uint16_t)two;
  }
}

}  // namespace gp
