// The norms around a block, with its gate and the residual, for gfx950:
//   u = norm_in(x) * w_in + b_in   (or x)
//   r = scale * R + gate * u       (gate: one row of H per M / G rows)
//   y = norm_out(r) * w_out + b_out
// norm is v / sqrt(mean(v^2) + eps), or (v - mean) / sqrt(var + eps). Bound by
// memory: each of x, R, r and y crosses HBM once. A row is held in registers
// between its reductions by WPR waves, 8 C columns a lane, so nothing is read
// twice; y is taken from r before r is rounded. Everything between the loads and
// the one rounding of each output is fp32; a layer norm takes the mean first and
// the squares of the centred values after it, which a mean far from zero does not
// spoil. A workgroup takes consecutive rows and keeps the columns' parameters in
// registers for all of them.
#pragma once

#include "gp_common.hpp"

namespace gp {

enum Norm : int { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };

struct NormArgs {
  const char *x, *res;                      // [M][H]; res null: no residual
  const float *w_in, *b_in, *gate, *w_out, *b_out;   // null: ones, zeros; gate [G][H]
  char *r, *y;                              // [M][H]; either null: not stored
  float scale, eps;
  uint32_t H, gate_rows, wg_rows;           // rows per gate row, rows per workgroup
  uint64_t M;
  int kin, kout;                            // Norm
};

// 8 elements of a 16-bit type <-> fp32
template <int DT>
__device__ __forceinline__ void widen8(v4i v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = widen16<DT>((uint32_t)v[i / 2], i & 1);
}
template <int DT>
__device__ __forceinline__ v4i narrow8(const float (&f)[8]) {
  const v2i lo = pack_out4<DT>(v4f{f[0], f[1], f[2], f[3]}), hi = pack_out4<DT>(v4f{f[4], f[5], f[6], f[7]});
  return v4i{lo[0], lo[1], hi[0], hi[1]};
}
// 8 floats of a vector over the columns, or the value it has where it is absent
__device__ __forceinline__ void load8(const float* p, uint32_t col, bool on, float absent, float (&f)[8]) {
  if (p && on) {
    const v4f a = *(const v4f*)(p + col), b = *(const v4f*)(p + col + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = absent;
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sums of N values over the WPR waves of a row, in the same order on every run. Of two
// halves of `red` consecutive sums take turns, so that one barrier each is enough:
// a half is written again only after the barrier of the sum between.
template <int WPR, int N>
struct RowSum {
  float* red;   // LDS [2][16][N]
  int wave, turn;
  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (WPR > 1) {
      float* half = red + turn * (16 * N);
      turn ^= 1;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((threadIdx.x & 63) == 0) half[wave * N + i] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = half[i];
        for (int w = 1; w < WPR; ++w) v[i] += half[w * N + i];
      }
    }
  }
};

constexpr int norm_threads(int wpr) { return wpr < 4 ? 256 : 64 * wpr; }

// Normalises the row v in place; the reciprocal root.
template <int WPR, int C>
__device__ __forceinline__ float normalize_row(int kind, float (&v)[C][8], const bool (&on)[C], float h, float eps,
                                               RowSum<WPR, 1>& sum) {
  float s[1] = {0.f};
  if (kind == NORM_LAYER) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += v[c][i];
    sum(s);
    const float mean = s[0] / h;   // exact for a row of one value, which then leaves zeros
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = on[c] ? v[c][i] - mean : 0.f;
    s[0] = 0.f;
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] = fmaf(v[c][i], v[c][i], s[0]);
  sum(s);
  const float rs = 1.f / sqrtf(s[0] / h + eps);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] *= rs;
  return rs;
}

template <int DT, int WPR, int C>
__global__ __launch_bounds__(norm_threads(WPR)) void norm_kernel(NormArgs p) {
  constexpr int T = 64 * WPR, RPW = norm_threads(WPR) / T;   // threads of a row, rows at a time
  constexpr bool KEEP = WPR * C < 32;   // parameters in registers (16 waves have 128 a lane)
  __shared__ float red[2 * 16];
  const int t = threadIdx.x % T;
  const uint32_t H = p.H;
  const float h = (float)H;
  RowSum<WPR, 1> sum{red, (int)threadIdx.x >> 6, 0};
  uint32_t col[C];
  bool on[C];
  float a[KEEP ? C : 1][8], b[KEEP ? C : 1][8], wo[KEEP ? C : 1][8], bo[KEEP ? C : 1][8];
  // gate * (n w_in + b_in) = n a + b
  auto load_in = [&](uint64_t g, int c, float (&av)[8], float (&bv)[8]) GP_INLINE {
    float gv[8];
    load8(p.w_in, col[c], on[c], 1.f, av);
    load8(p.b_in, col[c], on[c], 0.f, bv);
    load8(p.gate ? p.gate + g * H : nullptr, col[c], on[c], 1.f, gv);
#pragma unroll
    for (int i = 0; i < 8; ++i) av[i] *= gv[i], bv[i] *= gv[i];
  };
  auto load_out = [&](int c, float (&wv)[8], float (&bv)[8]) GP_INLINE {
    load8(p.w_out, col[c], on[c], 1.f, wv);
    load8(p.b_out, col[c], on[c], 0.f, bv);
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = (c * T + t) * 8u;
    on[c] = col[c] < H;
    if constexpr (KEEP) load_out(c, wo[c], bo[c]);
  }
  const uint64_t m0 = (uint64_t)blockIdx.x * p.wg_rows, m1 = min(m0 + p.wg_rows, p.M);
  uint64_t gate = 0, gate_end = 0;   // the gate row, and the row at which it changes
  v4i xv[C], rv[C];
  auto load = [&](uint64_t m) GP_INLINE {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const size_t off = (m * H + col[c]) * 2;
      xv[c] = on[c] && m < m1 ? *(const v4i*)(p.x + off) : v4i{0, 0, 0, 0};
      rv[c] = p.res && on[c] && m < m1 ? *(const v4i*)(p.res + off) : v4i{0, 0, 0, 0};
    }
  };
  uint64_t m = m0 + threadIdx.x / T;
  load(m);
  for (; m < m1; m += RPW) {
    if (m >= gate_end) {
      gate = m / p.gate_rows;
      gate_end = (gate + 1) * p.gate_rows;
      if constexpr (KEEP)
#pragma unroll
        for (int c = 0; c < C; ++c) load_in(gate, c, a[c], b[c]);
    }
    float v[C][8], r[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      widen8<DT>(xv[c], v[c]);
      widen8<DT>(rv[c], r[c]);
    }
    load(m + RPW);   // the next row's, while this one is reduced
    if (p.kin != NORM_NONE) normalize_row<WPR, C>(p.kin, v, on, h, p.eps, sum);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      constexpr auto at = [](int k) GP_INLINE { return KEEP ? k : 0; };
      if constexpr (!KEEP) load_in(gate, c, a[0], b[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        r[c][i] = on[c] ? fmaf(v[c][i], a[at(c)][i], b[at(c)][i]) + (p.res ? p.scale * r[c][i] : 0.f) : 0.f;
    }
    if (p.r)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (on[c]) *(v4i*)(p.r + (m * H + col[c]) * 2) = narrow8<DT>(r[c]);
    if (p.y) {
      normalize_row<WPR, C>(p.kout, r, on, h, p.eps, sum);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        constexpr auto at = [](int k) GP_INLINE { return KEEP ? k : 0; };
        if constexpr (!KEEP) load_out(c, wo[0], bo[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[c][i] = fmaf(r[c][i], wo[at(c)][i], bo[at(c)][i]);
        if (on[c]) *(v4i*)(p.y + (m * H + col[c]) * 2) = narrow8<DT>(r[c]);
      }
    }
  }
}

// ---- backward ----
// With n = norm_out(r), n1 = norm_in(x) (or x):
//   d = dy * w_out,   t = dr + rs (d - n mean(d n) [- mean(d) for a layer norm])
//   dR = scale t,     e = gate t w_in,   dx = rs1 (e - n1 mean(e n1) [- mean(e)])
// and over the rows, with T1 = sum t n1 and T0 = sum t within each gate row,
//   dw_out = sum dy n, db_out = sum dy, dgate = w_in T1 + b_in T0,
//   dw_in = sum gate T1, db_in = sum gate T0,
// so that four column sums serve all five parameters. A workgroup adds them up over
// its rows in fp32 (in registers, or in LDS for the longest rows, where a thread
// alone touches its columns) and stores them once; norm_sums_kernel adds the
// workgroups' sums in a fixed order. The statistics are taken again from x and r,
// which are read anyway.
struct NormGradArgs {
  const char *dy, *dr, *x, *r;              // [M][H]; dy null: no norm_out, dr null: none; x, r null: not needed
  const float *w_in, *gate, *w_out;
  char *dx, *dres;                          // either null: not stored
  float* part;                              // [workgroups][4][H]: dy n, dy, t n1, t
  float scale, eps;
  uint32_t H, gate_rows, wg_rows, wgs_per_gate;
  uint32_t sums;                            // bit i: sum i is wanted
  int kin, kout;
};

template <int WPR, int C>
__device__ __forceinline__ void normalize_grad(int kind, float (&d)[C][8], const float (&n)[C][8], const bool (&on)[C],
                                               float rs, float inv_h, RowSum<WPR, 2>& sum) {
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[0] = fmaf(d[c][i], n[c][i], s[0]);
      s[1] += d[c][i];
    }
  sum(s);
  const float along = s[0] * inv_h, mean = kind == NORM_LAYER ? s[1] * inv_h : 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) d[c][i] = on[c] ? rs * (d[c][i] - mean - n[c][i] * along) : 0.f;
}

constexpr int norm_grad_threads(int wpr) { return wpr < 4 ? 256 : 64 * wpr; }
// sums 2 and 3 in LDS: 16 waves have 128 registers a lane
constexpr bool norm_grad_lds(int wpr, int c) { return wpr * c >= 32; }

template <int DT, int WPR, int C>
__global__ __launch_bounds__(norm_grad_threads(WPR)) void norm_grad_kernel(NormGradArgs p) {
  constexpr int TH = norm_grad_threads(WPR), T = 64 * WPR, RPW = TH / T;
  constexpr bool LDS = norm_grad_lds(WPR, C);
  constexpr int NREG = LDS ? 2 : 4;
  __shared__ float red1[2 * 16], red2[2 * 16 * 2];
  __shared__ __attribute__((aligned(16))) v4f far[LDS ? 2 * C * T * 2 : 1];
  __shared__ float fold[RPW > 1 ? T * 8 : 1];
  const int t = threadIdx.x % T, grp = threadIdx.x / T;
  const uint32_t H = p.H;
  const float h = (float)H, inv_h = 1.f / h;
  RowSum<WPR, 1> sum1{red1, (int)threadIdx.x >> 6, 0};
  RowSum<WPR, 2> sum2{red2, (int)threadIdx.x >> 6, 0};
  const uint64_t g = blockIdx.x / p.wgs_per_gate;
  const uint64_t m0 = g * p.gate_rows + (uint64_t)(blockIdx.x % p.wgs_per_gate) * p.wg_rows;
  const uint64_t m1 = min(m0 + p.wg_rows, (g + 1) * (uint64_t)p.gate_rows);
  uint32_t col[C];
  bool on[C];
  float acc[NREG][C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = (c * T + t) * 8u;
    on[c] = col[c] < H;
#pragma unroll
    for (int k = 0; k < NREG; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[k][c][i] = 0.f;
  }
  auto far_at = [&](int k, int c, int h) GP_INLINE -> v4f& { return far[(((k - 2) * C + c) * 2 + h) * T + t]; };
  if constexpr (LDS)
#pragma unroll
    for (int k = 2; k < 4; ++k)
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) far_at(k, c, h) = v4f{0.f, 0.f, 0.f, 0.f};
  auto add = [&](auto k_c, int c, const float (&v)[8]) GP_INLINE {
    constexpr int k = decltype(k_c)::value;
    if constexpr (k < NREG) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[k][c][i] += v[i];
    } else {
      far_at(k, c, 0) += v4f{v[0], v[1], v[2], v[3]};
      far_at(k, c, 1) += v4f{v[4], v[5], v[6], v[7]};
    }
  };
  for (uint64_t m = m0 + grp; m < m1; m += RPW) {
    float d[C][8], n[C][8];
    v4i xv[C], rv[C], dv[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const size_t off = (m * H + col[c]) * 2;
      const v4i z = v4i{0, 0, 0, 0};
      rv[c] = p.dy && on[c] ? *(const v4i*)(p.r + off) : z;
      dv[c] = p.dy && on[c] ? *(const v4i*)(p.dy + off) : z;
      if constexpr (!LDS) xv[c] = p.x && on[c] ? *(const v4i*)(p.x + off) : z;
    }
    float rs = 0.f;
    if (p.dy) {
#pragma unroll
      for (int c = 0; c < C; ++c) widen8<DT>(rv[c], n[c]);
      rs = normalize_row<WPR, C>(p.kout, n, on, h, p.eps, sum1);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float w[8], v[8];
        widen8<DT>(dv[c], d[c]);
        if (p.sums & 2u) add(std::integral_constant<int, 1>{}, c, d[c]);
        if (p.sums & 1u) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = d[c][i] * n[c][i];
          add(std::integral_constant<int, 0>{}, c, v);
        }
        load8(p.w_out, col[c], on[c], 1.f, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[c][i] *= w[i];
      }
      normalize_grad<WPR, C>(p.kout, d, n, on, rs, inv_h, sum2);
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) d[c][i] = 0.f;
    }
    if (p.dr)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float v[8];
        widen8<DT>(on[c] ? *(const v4i*)(p.dr + (m * H + col[c]) * 2) : v4i{0, 0, 0, 0}, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[c][i] += v[i];
      }
    if (p.dres)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = p.scale * d[c][i];
        if (on[c]) *(v4i*)(p.dres + (m * H + col[c]) * 2) = narrow8<DT>(v);
      }
    if (!p.dx && !(p.sums & 12u)) continue;
    float rs1 = 0.f;
    if (p.x) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if constexpr (LDS) xv[c] = on[c] ? *(const v4i*)(p.x + (m * H + col[c]) * 2) : v4i{0, 0, 0, 0};
        widen8<DT>(xv[c], n[c]);
      }
      if (p.kin != NORM_NONE) rs1 = normalize_row<WPR, C>(p.kin, n, on, h, p.eps, sum1);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (p.sums & 8u) add(std::integral_constant<int, 3>{}, c, d[c]);
      if (p.sums & 4u) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = d[c][i] * n[c][i];
        add(std::integral_constant<int, 2>{}, c, v);
      }
    }
    if (!p.dx) continue;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float w[8], gv[8];
      load8(p.w_in, col[c], on[c], 1.f, w);
      load8(p.gate ? p.gate + g * H : nullptr, col[c], on[c], 1.f, gv);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[c][i] *= gv[i] * w[i];
    }
    if (p.kin != NORM_NONE) normalize_grad<WPR, C>(p.kin, d, n, on, rs1, inv_h, sum2);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (on[c]) *(v4i*)(p.dx + (m * H + col[c]) * 2) = narrow8<DT>(d[c]);
  }
  // the workgroup's sums; where it ran several rows at a time, theirs in order
  static_for<0, 4>([&](auto k_c) GP_INLINE {
    constexpr int k = decltype(k_c)::value;
    if (!(p.sums >> k & 1u)) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float v[8];
      if constexpr (k < NREG) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = acc[k][c][i];
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[4 * h + i] = far_at(k, c, h)[i];
      }
      if constexpr (RPW > 1) {
        for (int q = 0; q < RPW; ++q) {
          if (grp == q)
#pragma unroll
            for (int i = 0; i < 8; ++i) fold[i * T + t] = (q ? fold[i * T + t] : 0.f) + v[i];
          __syncthreads();
        }
        if (grp == 0)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = fold[i * T + t];
        __syncthreads();
      }
      if (grp == 0 && on[c]) {
        float* o = p.part + ((size_t)blockIdx.x * 4 + k) * H + col[c];
        *(v4f*)o = v4f{v[0], v[1], v[2], v[3]};
        *(v4f*)(o + 4) = v4f{v[4], v[5], v[6], v[7]};
      }
    }
  });
}

// Sums of the workgroups' parts: 32 columns a workgroup (blockIdx.x), 32 of the
// parts at a time, then those in order. blockIdx.y: 0 dw_out, 1 db_out, 2 dw_in, 3
// db_in, 4 + g the gradient of gate row g.
struct NormSumsArgs {
  const float *part, *gate, *w_in, *b_in;
  float *dw_out, *db_out, *dw_in, *db_in, *dgate;   // null: not wanted
  uint32_t H, parts, wgs_per_gate;
};
__global__ __launch_bounds__(1024) inline void norm_sums_kernel(NormSumsArgs p) {
  __shared__ float red[2][32][33];
  const uint32_t kind = blockIdx.y, lane = threadIdx.x & 31, row = threadIdx.x >> 5, H = p.H;
  const uint32_t c = blockIdx.x * 32u + lane;
  float* const out = kind == 0 ? p.dw_out : kind == 1 ? p.db_out : kind == 2 ? p.dw_in : kind == 3 ? p.db_in : p.dgate;
  if (!out) return;
  float s = 0.f, s0 = 0.f;
  if (c < H) {
    const bool of_gate = kind >= 4;
    const uint32_t first = of_gate ? (kind - 4) * p.wgs_per_gate : 0u, last = of_gate ? first + p.wgs_per_gate : p.parts;
    const uint32_t k = of_gate ? 2u : kind;
    for (uint32_t q = first + row; q < last; q += 32) {
      const float v = p.part[((size_t)q * 4 + k) * H + c];
      if (kind == 2 || kind == 3) s = fmaf(p.gate ? p.gate[(size_t)(q / p.wgs_per_gate) * H + c] : 1.f, v, s);
      else s += v;
      if (of_gate && p.b_in) s0 += p.part[((size_t)q * 4 + 3) * H + c];
    }
  }
  red[0][row][lane] = s;
  red[1][row][lane] = s0;
  __syncthreads();
  if (row != 0 || c >= H) return;
  s = s0 = 0.f;
  for (int q = 0; q < 32; ++q) {
    s += red[0][q][lane];
    s0 += red[1][q][lane];
  }
  if (kind >= 4) out[(size_t)(kind - 4) * H + c] = fmaf(p.w_in ? p.w_in[c] : 1.f, s, p.b_in ? p.b_in[c] * s0 : 0.f);
  else out[c] = s;
}

}  // namespace gp
