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
// spoil. The grid is what the CUs hold at once; a workgroup takes every so-manyth
// row (the rows under way at a time then lie together: 8192 x 8192 94 us, in runs of rows
// of a workgroup's own 105), loads the next while it reduces one, and keeps the columns'
// parameters in registers. Measured (residual, RMS norm): 16384 x 4096 98 us, 5.5 TB/s; 777 x
// 7168 11.1 (4.0 TB/s: three or four rows after each other on a CU); one row of 4096 3.2.
#pragma once

#include "gp_common.hpp"

namespace gp {

enum Norm : int { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };

struct NormArgs {
  const char *x, *res;                      // [M][H]; res null: no residual
  const float *w_in, *b_in, *gate, *w_out, *b_out;   // null: ones, zeros; gate [G][H]
  char *r, *y;                              // [M][H]; either null: not stored
  float scale, eps;
  uint32_t H, gate_rows;                    // gate_rows: rows per gate row
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

// Sums of N values over the WPR waves of a row, in the same order on every run. Of two
// halves of `red` consecutive sums take turns, so that one barrier each is enough: a half
// is written again only after the barrier of the sum between.
template <int WPR>
struct RowSum {
  float (*red)[2][16];   // LDS [2][2][16]
  int wave, turn;
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (WPR > 1) {
      float(*half)[16] = red[turn];
      turn ^= 1;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((threadIdx.x & 63) == 0) half[i][wave] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v4f t = *(const v4f*)&half[i][0];
#pragma unroll
        for (int w = 4; w < WPR; w += 4) t += *(const v4f*)&half[i][w];
        v[i] = (t[0] + t[1]) + (t[2] + t[3]);
      }
    }
  }
};

constexpr int norm_threads(int wpr) { return wpr < 4 ? 256 : 64 * wpr; }

// Normalises the row v in place; the reciprocal root. What lanes past the row hold is
// kept out of the sums (a piece at a time: a select per element is a tenth of the
// arithmetic). The root is the hardware's, 1 ulp, of a value that is scaled up where it
// would take it for zero; the mean is the quotient rounded once, so that a row of one
// value leaves zeros.
template <int WPR, int C>
__device__ __forceinline__ float normalize_row(int kind, float (&v)[C][8], const bool (&on)[C], uint32_t H, float inv_h,
                                               float eps, RowSum<WPR>& sum) {
  float s[1] = {0.f};
  if (kind == NORM_LAYER) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float t = v[c][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) t += v[c][i];
      s[0] += on[c] ? t : 0.f;
    }
    sum(s);
    float mean = s[0] * inv_h;
    mean = fmaf(fmaf(-mean, (float)H, s[0]), inv_h, mean);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] -= mean;
    s[0] = 0.f;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float t = v[c][0] * v[c][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) t = fmaf(v[c][i], v[c][i], t);
    s[0] += on[c] ? t : 0.f;
  }
  sum(s);
  const float mean2 = fmaf(s[0], inv_h, eps);
  const float rs = mean2 < 0x1p-100f ? 0x1p32f * __builtin_amdgcn_rsqf(0x1p64f * mean2) : __builtin_amdgcn_rsqf(mean2);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] *= rs;
  return rs;
}

template <int DT, int WPR, int C, bool KEEP>
__global__ __launch_bounds__(norm_threads(WPR)) void norm_kernel(NormArgs p) {
  constexpr int T = 64 * WPR, RPW = norm_threads(WPR) / T;   // threads of a row, rows at a time
  __shared__ __attribute__((aligned(16))) float red[2][2][16];
  const int t = threadIdx.x % T;
  const uint32_t H = p.H;
  const float inv_h = 1.f / (float)H;
  RowSum<WPR> sum{red, (int)threadIdx.x >> 6, 0};
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
  const uint64_t m0 = (uint64_t)blockIdx.x * RPW, m1 = p.M, step = (uint64_t)gridDim.x * RPW;
  const float scale = p.res ? p.scale : 0.f;   // (without a residual r holds zeros)
  uint64_t gate = 0, gate_end = 0;   // the gate row, and the row at which it changes
  v4i xv[C], rv[C];
  auto load = [&](const char* from, uint64_t m, v4i (&v)[C]) GP_INLINE {
#pragma unroll
    for (int c = 0; c < C; ++c)
      v[c] = from && on[c] && m < m1 ? *(const v4i*)(from + (m * H + col[c]) * 2) : v4i{0, 0, 0, 0};
  };
  uint64_t m = m0 + threadIdx.x / T;
  load(p.x, m, xv);
  if constexpr (KEEP) load(p.res, m, rv);
  for (; m < m1; m += step) {
    if (m >= gate_end) {
      gate = m / p.gate_rows;
      gate_end = (gate + 1) * p.gate_rows;
      if constexpr (KEEP)
#pragma unroll
        for (int c = 0; c < C; ++c) load_in(gate, c, a[c], b[c]);
    }
    float v[C][8], r[C][8];
    if constexpr (!KEEP) load(p.res, m, rv);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      widen8<DT>(xv[c], v[c]);
      if constexpr (KEEP) widen8<DT>(rv[c], r[c]);
    }
    load(p.x, m + step, xv);   // the next row's, while this one is reduced
    if constexpr (KEEP) load(p.res, m + step, rv);
    if (p.kin != NORM_NONE) normalize_row<WPR, C>(p.kin, v, on, H, inv_h, p.eps, sum);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      constexpr auto at = [](int k) GP_INLINE { return KEEP ? k : 0; };
      if constexpr (!KEEP) {
        widen8<DT>(rv[c], r[c]);
        load_in(gate, c, a[0], b[0]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        r[c][i] = fmaf(scale, r[c][i], fmaf(v[c][i], a[at(c)][i], b[at(c)][i]));
    }
    if (p.r)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (on[c]) *(v4i*)(p.r + (m * H + col[c]) * 2) = narrow8<DT>(r[c]);
    if (p.y) {
      normalize_row<WPR, C>(p.kout, r, on, H, inv_h, p.eps, sum);
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
// so that four column sums serve all five parameters. A workgroup adds them up over its
// rows (every so-manyth of one gate row) in fp32, in registers, or in LDS for the longest
// rows, where a thread alone touches its columns, and stores them once; norm_sums_kernel
// adds the workgroups' sums in a fixed order. The statistics are taken again from x and r,
// which are read anyway. IN: there is a norm_in or a gate; without them dx is t, and x is
// not read. Measured, bound by HBM: 16384 x 4096, a gate per sequence and a layer norm, 169 us
// (805 MB at 4.8 TB/s, the sums' launch among them).
struct NormGradArgs {
  const char *dy, *dr, *x, *r;              // [M][H]; dy null: no norm_out, dr null: none; x, r null: not needed
  const float *w_in, *gate, *w_out;
  char *dx, *dres;                          // either null: not stored
  float* part;                              // [workgroups][4][H]: dy n, dy, t n1, t
  float scale, eps;
  uint32_t H, gate_rows, wgs_per_gate;
  uint32_t sums;                            // bit i: sum i is wanted
  int kin, kout;
};

template <int WPR, int C>
__device__ __forceinline__ void normalize_grad(int kind, float (&d)[C][8], const float (&n)[C][8], const bool (&on)[C],
                                               float rs, float inv_h, RowSum<WPR>& sum) {
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float t = 0.f, u = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t = fmaf(d[c][i], n[c][i], t);
      u += d[c][i];
    }
    s[0] += on[c] ? t : 0.f;
    s[1] += on[c] ? u : 0.f;
  }
  sum(s);
  const float along = -rs * (s[0] * inv_h), shift = kind == NORM_LAYER ? -rs * (s[1] * inv_h) : 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) d[c][i] = fmaf(n[c][i], along, fmaf(d[c][i], rs, shift));
}

// sums 2 and 3 in LDS, parameters read again for each row: 16 waves have 128 registers a lane
constexpr bool norm_grad_lds(int wpr, int c) { return wpr * c >= 32; }

template <int DT, int WPR, int C, bool IN>
__global__ __launch_bounds__(norm_threads(WPR)) void norm_grad_kernel(NormGradArgs p) {
  constexpr int TH = norm_threads(WPR), T = 64 * WPR, RPW = TH / T;
  constexpr bool LDS = norm_grad_lds(WPR, C), KEEP = !LDS;
  constexpr int NSUM = IN ? 4 : 2, NREG = LDS && IN ? 2 : NSUM, K = KEEP ? C : 1;
  __shared__ __attribute__((aligned(16))) float red[2][2][16];
  __shared__ __attribute__((aligned(16))) v4f far[NREG < NSUM ? 2 * C * T * 2 : 1];
  __shared__ float fold[RPW > 1 ? T * 8 : 1];
  const int t = threadIdx.x % T, grp = threadIdx.x / T;
  const uint32_t H = p.H;
  const float inv_h = 1.f / (float)H;
  RowSum<WPR> sum{red, (int)threadIdx.x >> 6, 0};
  const uint64_t g = blockIdx.x / p.wgs_per_gate;
  const uint64_t m1 = (g + 1) * (uint64_t)p.gate_rows, step = (uint64_t)p.wgs_per_gate * RPW;
  uint32_t col[C];
  bool on[C];
  float acc[NREG][C][8], wo[K][8], wi[K][8];
  auto load_in = [&](int c, float (&w)[8]) GP_INLINE {   // gate * w_in
    float gv[8];
    load8(p.w_in, col[c], on[c], 1.f, w);
    load8(p.gate ? p.gate + g * H : nullptr, col[c], on[c], 1.f, gv);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] *= gv[i];
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = (c * T + t) * 8u;
    on[c] = col[c] < H;
    if constexpr (KEEP) {
      load8(p.w_out, col[c], on[c], 1.f, wo[c]);
      if constexpr (IN) load_in(c, wi[c]);
    }
#pragma unroll
    for (int k = 0; k < NREG; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[k][c][i] = 0.f;
  }
  auto far_at = [&](int k, int c, int h) GP_INLINE -> v4f& { return far[(((k - 2) * C + c) * 2 + h) * T + t]; };
  if constexpr (NREG < NSUM)
#pragma unroll
    for (int k = 2; k < 4; ++k)
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) far_at(k, c, h) = v4f{0.f, 0.f, 0.f, 0.f};
  // adds v (one) or v w to sum k
  auto add = [&](auto k_c, int c, const float (&v)[8], const float (&w)[8], bool one) GP_INLINE {
    constexpr int k = decltype(k_c)::value;
    if constexpr (k < NREG) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[k][c][i] = one ? acc[k][c][i] + v[i] : fmaf(v[i], w[i], acc[k][c][i]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v4f f = far_at(k, c, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = one ? f[i] + v[4 * h + i] : fmaf(v[4 * h + i], w[4 * h + i], f[i]);
        far_at(k, c, h) = f;
      }
    }
  };
  v4i xv[C], rv[C], dv[C], sv[C];
  auto load = [&](const char* from, uint64_t m, v4i (&v)[C]) GP_INLINE {
#pragma unroll
    for (int c = 0; c < C; ++c)
      v[c] = from && on[c] && m < m1 ? *(const v4i*)(from + (m * H + col[c]) * 2) : v4i{0, 0, 0, 0};
  };
  auto load_row = [&](uint64_t m) GP_INLINE {
    load(p.r, m, rv);
    load(p.dy, m, dv);
    if constexpr (KEEP) {
      load(p.dr, m, sv);
      if constexpr (IN) load(p.x, m, xv);
    }
  };
  uint64_t m = g * p.gate_rows + (uint64_t)(blockIdx.x % p.wgs_per_gate) * RPW + grp;
  if constexpr (KEEP) load_row(m);
  for (; m < m1; m += step) {
    float d[C][8], n[C][8];
    v4i s[C], x[C];   // of dr and x, as they were loaded
    if constexpr (!KEEP) load_row(m);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      widen8<DT>(rv[c], n[c]);
      widen8<DT>(dv[c], d[c]);
      if constexpr (KEEP) {
        s[c] = sv[c];
        if constexpr (IN) x[c] = xv[c];
      }
    }
    if constexpr (KEEP) load_row(m + step);   // the next row's, while this one is reduced
    if (p.dy) {
      const float rs = normalize_row<WPR, C>(p.kout, n, on, H, inv_h, p.eps, sum);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (p.sums & 2u) add(std::integral_constant<int, 1>{}, c, d[c], d[c], true);
        if (p.sums & 1u) add(std::integral_constant<int, 0>{}, c, d[c], n[c], false);
        if constexpr (!KEEP) load8(p.w_out, col[c], on[c], 1.f, wo[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[c][i] *= wo[KEEP ? c : 0][i];
      }
      normalize_grad<WPR, C>(p.kout, d, n, on, rs, inv_h, sum);
    }
    if (p.dr) {
      if constexpr (!KEEP) load(p.dr, m, s);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float v[8];
        widen8<DT>(s[c], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[c][i] += v[i];
      }
    }
    if (p.dres)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = p.scale * d[c][i];
        if (on[c]) *(v4i*)(p.dres + (m * H + col[c]) * 2) = narrow8<DT>(v);
      }
    if constexpr (IN) {
      float rs1 = 0.f;
      if (p.x) {
        if constexpr (!KEEP) load(p.x, m, x);
#pragma unroll
        for (int c = 0; c < C; ++c) widen8<DT>(x[c], n[c]);
        if (p.kin != NORM_NONE) rs1 = normalize_row<WPR, C>(p.kin, n, on, H, inv_h, p.eps, sum);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (p.sums & 8u) add(std::integral_constant<int, 3>{}, c, d[c], d[c], true);
        if (p.sums & 4u) add(std::integral_constant<int, 2>{}, c, d[c], n[c], false);
      }
      if (p.dx) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if constexpr (!KEEP) load_in(c, wi[0]);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[c][i] *= wi[KEEP ? c : 0][i];
        }
        if (p.kin != NORM_NONE) normalize_grad<WPR, C>(p.kin, d, n, on, rs1, inv_h, sum);
      }
    }
    if (p.dx)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (on[c]) *(v4i*)(p.dx + (m * H + col[c]) * 2) = narrow8<DT>(d[c]);
  }
  // the workgroup's sums; where it ran several rows at a time, theirs in order
  static_for<0, NSUM>([&](auto k_c) GP_INLINE {
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

// Sums of the workgroups' parts: 64 columns a workgroup (blockIdx.x), four a lane, 64 of
// the parts at a time, then those in order. blockIdx.y: 0 dw_out, 1 db_out, 2 dw_in, 3
// db_in, 4 + g the gradient of gate row g.
struct NormSumsArgs {
  const float *part, *gate, *w_in, *b_in;
  float *dw_out, *db_out, *dw_in, *db_in, *dgate;   // null: not wanted
  uint32_t H, parts, wgs_per_gate;
};
static __global__ __launch_bounds__(1024) void norm_sums_kernel(NormSumsArgs p) {
  __shared__ __attribute__((aligned(16))) v4f red[2][64][16];
  const uint32_t kind = blockIdx.y, lane = threadIdx.x & 15, row = threadIdx.x >> 4, H = p.H;
  const uint32_t c = blockIdx.x * 64u + 4 * lane;
  float* const out = kind == 0 ? p.dw_out : kind == 1 ? p.db_out : kind == 2 ? p.dw_in : kind == 3 ? p.db_in : p.dgate;
  if (!out) return;
  const v4f zero = v4f{0.f, 0.f, 0.f, 0.f};
  v4f s = zero, s0 = zero;
  const bool of_gate = kind >= 4;
  if (c < H) {
    const uint32_t first = of_gate ? (kind - 4) * p.wgs_per_gate : 0u, last = of_gate ? first + p.wgs_per_gate : p.parts;
    const uint32_t k = of_gate ? 2u : kind;
#pragma unroll 4
    for (uint32_t q = first + row; q < last; q += 64) {
      v4f v = *(const v4f*)(p.part + ((size_t)q * 4 + k) * H + c);
      if ((kind == 2 || kind == 3) && p.gate) v *= *(const v4f*)(p.gate + (size_t)(q / p.wgs_per_gate) * H + c);
      s += v;
      if (of_gate && p.b_in) s0 += *(const v4f*)(p.part + ((size_t)q * 4 + 3) * H + c);
    }
  }
  red[0][row][lane] = s;
  red[1][row][lane] = s0;
  __syncthreads();
  const uint32_t x = threadIdx.x, col = blockIdx.x * 64u + x;   // a lane a column
  if (x >= 64 || col >= H) return;
  float a = 0.f, a0 = 0.f;
#pragma unroll 8
  for (int q = 0; q < 64; ++q) {
    a += red[0][q][x / 4][x % 4];
    a0 += red[1][q][x / 4][x % 4];
  }
  if (of_gate) out[(size_t)(kind - 4) * H + col] = fmaf(p.w_in ? p.w_in[col] : 1.f, a, p.b_in ? p.b_in[col] * a0 : 0.f);
  else out[col] = a;
}

}  // namespace gp
