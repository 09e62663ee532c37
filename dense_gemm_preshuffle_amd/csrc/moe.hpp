// A mixture-of-experts layer for a few tokens, for gfx950, in three launches:
//   route   l = x Wr^T, p = softmax(l) or sigmoid(l), the k experts of largest p (+
//           bias) of each token, their weights g
//   up      h[p] = g_j act(x Wg_e^T) * (x Wu_e^T)    for each pair p = (token, choice j)
//   down    y = residual + sum over j of h[p] Wd_e^T
// Bound by reading the chosen experts' weights from HBM, once each: a workgroup owns an
// expert's NB column blocks and runs all its tokens through them, found in a list that
// it makes from the choices itself. Nothing of an expert without tokens is read.
#pragma once

#include "gp_common.hpp"

namespace gp {

// ---- the router ----
// Sums in 64 bits: which of two experts with close scores is chosen then does not
// depend on the order of a sum (the products of 16-bit values are exact; an fp32 sum
// of 4096 is off by 1e-6, as far as two of 128 scores lie apart once in some
// thousand tokens). A workgroup takes EB experts and TB tokens; the last of a token
// block to finish chooses for its tokens, a wave for each. Bound by latency: one token,
// 8 of 64 experts, H 2048 5.8 us (0.26 MB; 2 of them launch, 2 the arrival and the choice).
struct RouteArgs {
  const char *x, *wr;       // [M][H], [E][H]
  const float* bias;        // [E] added for the choice alone, or null
  double* logits;           // [M][E]
  uint32_t* cnt;            // [token blocks]: zero before and after
  int32_t* ids;             // [M][k], by falling score
  float* gates;             // [M][k]
  uint32_t M, E, H, k;
  int sigmoid, normalize;
  float scale;
};

constexpr uint32_t kMaxExperts = 512;

// The k experts of token m, by one wave: lane l has experts l, l + 64, ... (NE of them).
// Each round takes the largest key of the wave; a key orders as its double does, with NaN
// (1) below every number and 0 for an expert that is not there or chosen already.
// Scores that the result does not need are not taken: without a bias the logits order
// the experts as their scores do (and do not saturate), and in normalised softmax
// weights the sum over all experts cancels.
template <int NE>
__device__ __forceinline__ void choose_experts(const RouteArgs& p, uint32_t m, uint32_t lane) {
  auto key = [](double v) GP_INLINE -> uint64_t {
    if (!(v == v)) return 1;
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);   // (-0 as 0)
    return u >> 63 ? ~u : u | 1ull << 63;
  };
  double l[NE];
  uint64_t keys[NE];
  double top = -__builtin_inf();
  bool nan = false;
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    l[j] = 0.0;
    keys[j] = 0;
    const uint32_t e = lane + 64u * j;
    if (e >= p.E) continue;
    const uint64_t u = __hip_atomic_load((const uint64_t*)p.logits + (size_t)m * p.E + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    l[j] = __builtin_bit_cast(double, u);
    keys[j] = key(l[j]);
    nan = nan || keys[j] == 1;
    top = fmax(top, l[j]);
  }
  // (fmax passes over NaN, but the sum over the experts would not: one makes every softmax
  // score NaN, also where that sum cancels and the expert is not chosen)
  if (!p.sigmoid) {
    top = wave_reduce64(top, [](double a, double b) GP_INLINE { return fmax(a, b); });
    if (__ballot(nan)) top = __builtin_nan("");
  }
  // (softmax: the score times the sum over the experts)
  auto score = [&](double v) GP_INLINE { return p.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - top); };
  double sum = 1.0;
  if (p.bias || (!p.sigmoid && !p.normalize)) {
    double s[NE], mine = 0.0;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      s[j] = keys[j] ? score(l[j]) : 0.0;
      mine += s[j];
    }
    if (!p.sigmoid) sum = wave_sum64(mine);
    if (p.bias)
#pragma unroll
      for (int j = 0; j < NE; ++j)
        if (keys[j]) keys[j] = key(s[j] / sum + (double)p.bias[lane + 64 * j]);
  }
  uint64_t best = 0;
  uint32_t at = 0;   // the lane's largest key and its j
  auto lane_best = [&]() GP_INLINE {
    best = keys[0];
    at = 0;
#pragma unroll
    for (int j = 1; j < NE; ++j)
      if (keys[j] > best) best = keys[j], at = j;
  };
  lane_best();
  uint32_t rank[NE];
#pragma unroll
  for (int j = 0; j < NE; ++j) rank[j] = ~0u;
  for (uint32_t c = 0; c < p.k; ++c) {
    const uint64_t most = wave_reduce64(best, [](uint64_t a, uint64_t b) GP_INLINE { return a > b ? a : b; });
    // ties go to the lowest expert: the lowest j, then the lowest lane
    uint64_t who = 0;
    uint32_t j0 = 0;
    for (; j0 < (uint32_t)NE; ++j0)
      if ((who = __ballot(best == most && at == j0))) break;
    if (lane == (uint32_t)__builtin_ctzll(who)) {
#pragma unroll
      for (int j = 0; j < NE; ++j)
        if ((uint32_t)j == j0) {
          keys[j] = 0;
          rank[j] = c;
        }
      lane_best();
    }
  }
  double mine = 0.0;   // the lane's chosen scores
#pragma unroll
  for (int j = 0; j < NE; ++j)
    if (rank[j] != ~0u) {
      l[j] = score(l[j]);
      mine += l[j];
    }
  const double total = p.normalize ? wave_sum64(mine) : sum;
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    if (rank[j] == ~0u) continue;
    p.ids[(size_t)m * p.k + rank[j]] = (int32_t)(lane + 64 * j);
    p.gates[(size_t)m * p.k + rank[j]] = (float)(l[j] / total * (double)p.scale);
  }
}

// Sums of N values (a power of two up to 16) over each row of 16 lanes: a step hands one
// half of the values to the other half of the lanes and adds what comes back, so that N
// values take N - 1 exchanges and not 4 N. The lane ends up with value lane % 16 /
// (16 / N) of its row.
template <int N>
__device__ __forceinline__ double row_sums(double (&v)[N], uint32_t lane) {
  auto step = [&](auto n_c, auto ctrl_c, uint32_t bit) GP_INLINE {
    constexpr int n = decltype(n_c)::value, ctrl = decltype(ctrl_c)::value;
    auto other = [](double x) GP_INLINE { return __builtin_bit_cast(double, dpp64<ctrl>(__builtin_bit_cast(uint64_t, x))); };
    if constexpr (n > 1) {
      const bool up = lane & bit;
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const double keep = up ? v[i + n / 2] : v[i], give = up ? v[i] : v[i + n / 2];
        v[i] = keep + other(give);
      }
    } else {
      v[0] += other(v[0]);
    }
  };
  constexpr auto left = [](int s) { return N >> s > 1 ? N >> s : 1; };
  step(std::integral_constant<int, left(0)>{}, std::integral_constant<int, kDppRowMirror>{}, 8);
  step(std::integral_constant<int, left(1)>{}, std::integral_constant<int, kDppHalfRowMirror>{}, 4);
  step(std::integral_constant<int, left(2)>{}, std::integral_constant<int, kDppSwapQuadHalves>{}, 2);
  step(std::integral_constant<int, left(3)>{}, std::integral_constant<int, kDppSwapPairs>{}, 1);
  return v[0];
}

template <int DT, int TB, int EB>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs p) {
  constexpr int N = TB * EB;
  __shared__ double red[16][N];   // of each row of 16 lanes
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t e0 = blockIdx.x * EB, m0 = blockIdx.y * TB;
  double acc[N] = {};
#pragma unroll TB == 1 ? 2 : 1
  for (uint32_t c = tid; c < p.H / 8; c += 256) {
    v4i xv[TB], wv[EB];
#pragma unroll
    for (int t = 0; t < TB; ++t) xv[t] = m0 + t < p.M ? *(const v4i*)(p.x + ((size_t)(m0 + t) * p.H + 8 * c) * 2) : v4i{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < EB; ++e) wv[e] = e0 + e < p.E ? *(const v4i*)(p.wr + ((size_t)(e0 + e) * p.H + 8 * c) * 2) : v4i{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      double w[EB];
#pragma unroll
      for (int e = 0; e < EB; ++e) w[e] = (double)widen16<DT>((uint32_t)wv[e][i / 2], i & 1);
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const double x = (double)widen16<DT>((uint32_t)xv[t][i / 2], i & 1);
#pragma unroll
        for (int e = 0; e < EB; ++e) acc[t * EB + e] = fma(x, w[e], acc[t * EB + e]);
      }
    }
  }
  const double row = row_sums<N>(acc, lane);
  if (lane % (16 / N) == 0) red[tid / 16][lane % 16 / (16 / N)] = row;
  __syncthreads();
  if (tid < N) {
    double v = 0.0;
#pragma unroll
    for (int r = 0; r < 16; ++r) v += red[r][tid];
    const uint32_t t = tid / EB, e = tid % EB;
    if (m0 + t < p.M && e0 + e < p.E)
      __hip_atomic_store((uint64_t*)p.logits + (size_t)(m0 + t) * p.E + e0 + e, __builtin_bit_cast(uint64_t, v),
                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  auto choose = [&](uint32_t m) GP_INLINE {
    if (p.E <= 64) choose_experts<1>(p, m, lane);
    else if (p.E <= 128) choose_experts<2>(p, m, lane);
    else if (p.E <= 256) choose_experts<4>(p, m, lane);
    else choose_experts<8>(p, m, lane);
  };
  if constexpr (TB == 1) {
    // one wave stores, arrives and chooses: no barrier (as last_to_arrive otherwise)
    if (wave != 0) return;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the logits are stored
    uint32_t before = 0;
    if (lane == 0) before = __hip_atomic_fetch_add(p.cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if ((uint32_t)__builtin_amdgcn_readfirstlane((int)before) != gridDim.x - 1) return;
    if (lane == 0) __hip_atomic_store(p.cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    choose(m0);
  } else {
    __shared__ uint32_t word;
    if (!last_to_arrive(p.cnt + blockIdx.y, gridDim.x, &word)) return;
    for (uint32_t t = wave; t < TB; t += 4)
      if (m0 + t < p.M) choose(m0 + t);
  }
}

// ---- the experts' products ----
struct MoeArgs {
  const char* a;            // up: x [M][Ka]; down: h [pairs][Ka]
  const char* b;            // the experts' preshuffled weights (up: gate and up blocks alternating), expert_bytes each
  size_t expert_bytes;
  const int32_t* ids;       // [pairs]; outside [0, E): no expert, the pair adds nothing
  char* h;                  // up: [pairs][F]
  const float* gates;       // up: [pairs]
  const char* res;          // down: [M][F], or null
  char* y;                  // down: [M][F]
  float* part;              // down: [pairs][F]
  uint32_t* cnt;            // down: [column groups]: zero before and after
  uint32_t M, k, E, F;      // F: output columns
  uint32_t Ka, Kb;          // bytes of K per row of a, and of the weights (whole 128-byte chunks, zeros past Ka)
  uint32_t slots;           // pairs where they are no more than the experts (a slot is then a pair), else the experts
  uint32_t cols;            // column groups
  int act;
};

constexpr uint32_t kMaxPairs = 4096;

// The pairs of this workgroup's expert in list, in order, by the first wave; their
// number. Slots by pair: the first pair of an expert has it, the others none.
__device__ __forceinline__ uint32_t list_pairs(const MoeArgs& p, uint32_t slot, bool by_pair, uint32_t e, uint16_t* list) {
  const uint32_t pairs = p.M * p.k, lane = threadIdx.x & 63;
  uint32_t n = 0;
  if (e >= p.E) return 0;
  for (uint32_t q0 = 0; q0 < pairs; q0 += 64) {
    const uint32_t q = q0 + lane;
    const bool is = q < pairs && (uint32_t)p.ids[q] == e;
    const uint64_t mask = __ballot(is);
    if (by_pair && n == 0 && mask && q0 + (uint32_t)__builtin_ctzll(mask) != slot) return 0;
    if (is) list[n + __builtin_popcountll(mask & ((1ull << lane) - 1))] = (uint16_t)q;
    n += (uint32_t)__builtin_popcountll(mask);
  }
  return n;
}

// As ffn_small_kernel (ffn_small.hpp), on the rows of a list: NB 16-column blocks of
// weights a workgroup, K split over its WAVES waves in chunks of 64 elements, two
// groups of S chunks of weights in flight; x passes through a piece of LDS of the
// wave's own. XL: 16-byte loads of a per lane and chunk, 8 XL rows at a time; 0: one
// row. Longer lists take further turns, which find the weights in L2 or read them again.
// Measured: 33 tokens, 2 of 8 experts of 4096 x 14336, up 313 us (1.88 GB, 6.0 TB/s), down
// 145 (0.94 GB, 6.5 TB/s); one token, 8 of 64 of 2048 x 1024, up 13.2 (67 MB, 5.1 TB/s).
template <int DT, int XL, int NB, int WAVES, int S, bool UP>
__global__ __launch_bounds__(WAVES * 64) void moe_kernel(MoeArgs p) {
  constexpr bool ONE = XL == 0;
  constexpr int ROWS = ONE ? 1 : 8 * XL;
  constexpr int MB = (ROWS + 15) / 16;
  constexpr int OB = UP ? NB / 2 : NB;   // 16-column blocks of the output
  constexpr int NV = NB / OB;            // sums of an output
  constexpr int NQ = MB * NB;
  constexpr int XW = (ONE ? 2 : ROWS) * 128;
  constexpr int LDS = WAVES * (XW > NQ * 1024 ? XW : NQ * 1024);
  __shared__ __attribute__((aligned(16))) char lds[LDS];
  __shared__ uint16_t list[ONE ? 1 : kMaxPairs];
  __shared__ uint32_t count, word;

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, lane_lo = lane & 15, lane_hi = lane >> 4;
  const uint32_t Ka = p.Ka, Kb = p.Kb, pairs = p.M * p.k;
  const uint32_t slot = blockIdx.x / p.cols, bx = blockIdx.x % p.cols;
  const bool by_pair = p.slots == pairs;
  const uint32_t e = __builtin_amdgcn_readfirstlane(by_pair ? (uint32_t)p.ids[slot] : slot);
  // one token: a slot is a pair (an expert that stands twice is read twice)
  uint32_t n = e < p.E ? 1u : 0u;
  if constexpr (!ONE) {
    if (wave == 0) {
      const uint32_t l = list_pairs(p, slot, by_pair, e, list);
      if (lane == 0) count = l;
    }
    __syncthreads();
    n = __builtin_amdgcn_readfirstlane(count);
  }
  if (UP && n == 0) return;
  auto pair_at = [&](uint32_t r) GP_INLINE -> uint32_t { return ONE ? slot : list[r]; };

  const uint32_t blocks = p.F / 16, block0 = bx * OB;
  const uint32_t nblock = min((uint32_t)OB, blocks - block0);   // real blocks of this workgroup
  const uint32_t nchunk = Kb / 128;
  const uint32_t kc0 = wave * nchunk / WAVES, kc1 = (wave + 1) * nchunk / WAVES;
  const int groups = (int)((kc1 - kc0 + S - 1) / S);
  const __amdgpu_buffer_rsrc_t rb =
      make_rsrc(p.b + (n ? e : 0u) * p.expert_bytes + (size_t)block0 * (NV * 16) * Kb, nblock * (NV * 16) * Kb);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a, (UP ? p.M : pairs) * Ka);
  constexpr uint32_t kOOB = 0x80000000u;
  char* xw = lds + wave * XW;
  const uint32_t xcol = ONE ? 4 * lane : 16 * (lane & 7);

  for (uint32_t r0 = 0; r0 < n; r0 += ROWS) {
    const uint32_t rows = min((uint32_t)ROWS, n - r0);
    auto a_row = [&](uint32_t r) GP_INLINE -> uint32_t {   // offset of a list entry's row
      const uint32_t q = pair_at(r0 + r);
      return (UP ? q / p.k : q) * Ka;
    };
    uint32_t x_off[XL > 0 ? XL : 1];
    if constexpr (ONE) x_off[0] = lane < 32 ? a_row(0) + xcol : kOOB;
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const uint32_t r = 8 * i + (lane >> 3);
      x_off[i] = r < rows ? a_row(r) + xcol : kOOB;
    }
    v4i xr[2][S][XL > 0 ? XL : 1], bf[2][S][2][NB];
    v4f acc[MB][NB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = v4f{0.f, 0.f, 0.f, 0.f};
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
        const uint32_t off = (128 * k + xcol < Ka ? 0u : kOOB) | skip;
        if constexpr (ONE) xr[par][s][0][0] = buf_load4(ra, x_off[0] | off, 128 * k);
#pragma unroll
        for (int i = 0; i < XL; ++i) xr[par][s][i] = buf_load16(ra, x_off[i] | off, 128 * k);
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
            if (MB > 1 && 16u * mb >= rows) continue;   // uniform
            const int m = ONE ? 0 : (mb * 16 + lane_lo) % ROWS;
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
    __syncthreads();   // the sums take the place of the waves' rows
    v4f* red = (v4f*)lds;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) red[(wave * NQ + mb * NB + nb) * 64 + lane] = acc[mb][nb];
    __syncthreads();
    for (uint32_t q = (uint32_t)wave; q < MB * OB; q += WAVES) {
      const uint32_t mb = q / OB, ob = q % OB, row = mb * 16 + lane_lo;
      if (ob >= nblock || row >= rows) continue;
      v4f v[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        v[i] = red[(NV * q + i) * 64 + lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v[i] += red[(w * NQ + NV * q + i) * 64 + lane];
      }
      const uint32_t pair = pair_at(r0 + row), col = (block0 + ob) * 16 + 4 * lane_hi;
      if constexpr (UP) {
        // weighted here, so that the down product adds a token's experts up as they are,
        // and rounded to the type, as the matrix products take it (33 tokens in fp16 are off by
        // 0.00029 of their size, with an fp32 h by 0.00021; a second operand for the rest
        // would double the down product's instructions and its reads of h)
        v4f h;
        const float g = p.gates[pair];
        with_act(p.act, [&](auto act_c) GP_INLINE {
          constexpr int A = decltype(act_c)::value;
#pragma unroll
          for (int r = 0; r < 4; ++r) h[r] = g * (activate_ffn<A>(v[0][r]) * v[1][r]);
        });
        *(v2i*)(p.h + ((size_t)pair * p.F + col) * 2) = pack_out4<DT>(h);
      } else {
        const __amdgpu_buffer_rsrc_t rp = make_rsrc(p.part, pairs * p.F * 4);
        buf_store16_coh(__builtin_bit_cast(v4i, v[0]), rp, (pair * p.F + col) * 4);
      }
    }
    __syncthreads();   // before the next rows take the sums' place
  }
  if constexpr (!UP) {
    // the last workgroup of the columns adds up each token's experts, in the order of
    // its choices
    if (!last_to_arrive(p.cnt + bx, p.slots, &word)) return;
    const __amdgpu_buffer_rsrc_t rp = make_rsrc(p.part, pairs * p.F * 4);
    for (uint32_t i = tid; i < p.M * nblock * 4; i += WAVES * 64) {
      const uint32_t m = i / (nblock * 4), col = block0 * 16 + 4 * (i % (nblock * 4));
      v4f v = v4f{0.f, 0.f, 0.f, 0.f};
      for (uint32_t j = 0; j < p.k; ++j) {
        const uint32_t q = m * p.k + j;
        if ((uint32_t)p.ids[q] >= p.E) continue;
        v += __builtin_bit_cast(v4f, buf_load16_coh(rp, (q * p.F + col) * 4));
      }
      const size_t off = ((size_t)m * p.F + col) * 2;
      if (p.res) v += widen4<DT>(*(const v2i*)(p.res + off));
      *(v2i*)(p.y + off) = pack_out4<DT>(v);
    }
  }
}

// The down product of one token: its k experts' products are one of K = k Ka. WAVES waves
// split those chunks, so that a workgroup's columns are finished by itself: no partial
// products in memory and no arrival, which take the general form 3 us of 11 (8 experts of
// 2048 x 1024: 8.4 us, 4.0 TB/s; launch and the waves' join are 2.5 of them).
template <int DT, int NB, int WAVES, int S>
__global__ __launch_bounds__(WAVES * 64) void moe_down_one_kernel(MoeArgs p) {
  __shared__ __attribute__((aligned(16))) char lds[WAVES * NB * 1024];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, lane_lo = lane & 15, lane_hi = lane >> 4;
  const uint32_t Ka = p.Ka, Kb = p.Kb;
  const uint32_t block0 = blockIdx.x * NB, nblock = min((uint32_t)NB, p.F / 16 - block0);
  const uint32_t nchunk = Kb / 128, all = p.k * nchunk;
  const uint32_t c0 = wave * all / WAVES, c1 = (wave + 1) * all / WAVES;
  const int groups = (int)((c1 - c0 + S - 1) / S);
  const int id = (uint32_t)lane < p.k ? p.ids[lane] : -1;   // lane j: choice j
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a, p.k * Ka);
  constexpr uint32_t kOOB = 0x80000000u;
  char* xw = lds + wave * (NB * 1024);
  const uint32_t xcol = 4 * lane;
  int xr[2][S];
  v4i bf[2][S][2][NB];
  v4f acc[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) acc[nb] = v4f{0.f, 0.f, 0.f, 0.f};
  auto load = [&](auto par_c, int gr) GP_INLINE {
    constexpr int par = decltype(par_c)::value;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const uint32_t c = c0 + (uint32_t)gr * S + s, j = min(c / nchunk, p.k - 1), k = c - j * nchunk;
      const uint32_t e = (uint32_t)__builtin_amdgcn_readlane(id, (int)j);
      const bool is = c < c1 && e < p.E;   // (else zeros from an empty resource)
      const __amdgpu_buffer_rsrc_t rb =
          make_rsrc(p.b + (is ? e : 0u) * p.expert_bytes + (size_t)block0 * 16 * Kb, is ? nblock * 16 * Kb : 0u);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        bf[par][s][0][nb] = buf_load16_nt(rb, nb * 16 * Kb + lane * 16, k * 2048);
        bf[par][s][1][nb] = buf_load16_nt(rb, nb * 16 * Kb + lane * 16 + 1024, k * 2048);
      }
      xr[par][s] = buf_load4(ra, is && lane < 32 && 128 * k + xcol < Ka ? xcol : kOOB, j * Ka + 128 * k);
    }
  };
  auto compute = [&](auto par_c) GP_INLINE {
    constexpr int par = decltype(par_c)::value;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      *(int*)(xw + 4 * lane) = xr[par][s];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const v4i xf = *(const v4i*)(xw + (4 * t + lane_hi) * 16);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[nb] = mfma<DT>(&bf[par][s][t][nb], &xf, acc[nb]);
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
  // (each wave's sums take the place of its own x)
  v4f* red = (v4f*)lds;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) red[(wave * NB + nb) * 64 + lane] = acc[nb];
  __syncthreads();
  if (wave >= NB || (uint32_t)wave >= nblock || lane_lo != 0) return;
  v4f v = red[wave * 64 + lane];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) v += red[(w * NB + wave) * 64 + lane];
  const size_t off = ((block0 + wave) * 16 + 4 * lane_hi) * 2;
  if (p.res) v += widen4<DT>(*(const v2i*)(p.res + off));
  *(v2i*)(p.y + off) = pack_out4<DT>(v);
}

}  // namespace gp
