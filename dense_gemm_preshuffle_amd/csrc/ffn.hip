// Host side of the gated feed-forward product, its backward pass and the
// backward pass of a linear layer: validation, plans, workspaces, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/gemm_preshuffle.h"
#include "host.hpp"
#include "launch_gated.hpp"
#include "launch_rows.hpp"
#include "transpose.hpp"

namespace gp {
namespace {

bool half_type(int dtype) { return dtype == GP_BF16 || dtype == GP_F16; }

// 16-byte pieces of the preshuffled gated layout: block 2p is gate block p of
// the weights, block 2p + 1 up block p; K is filled up to kb64 64-byte blocks (a
// multiple of two) with zeros.
__global__ __launch_bounds__(256) void preshuffle_gated_kernel(const char* __restrict__ w, char* __restrict__ dst,
                                                               uint32_t kb64, uint32_t Ka, uint32_t F, uint32_t chunks) {
  const uint32_t x = blockIdx.x * 256u + threadIdx.x;
  if (x >= chunks) return;
  const uint32_t j = x & 15u, g = (x >> 4) & 3u, t = x >> 6;
  const uint32_t k0 = t % kb64, nb = t / kb64;
  const uint32_t row = (nb & 1u) * F + (nb >> 1) * 16u + j, col = 64u * k0 + 16u * g;
  *(v4i*)(dst + (size_t)x * 16u) = col < Ka ? *(const v4i*)(w + (size_t)row * Ka + col) : v4i{0, 0, 0, 0};
}

// ---- tiles ----
// Time of a product [M][K] x [K][N] on the tile kernel in us, by the model
//   start + rounds * (K tiles per range * step + ends) + ranges * join
// of its workgroups on 256 CUs. step: a 128-byte K tile; ends: filling the
// pipeline and storing the tile; join: writing a range's partial tile and the last
// workgroup's reading it (0: the tile is not split; a smaller one takes less
// time wherever CUs would idle). Two workgroups on a CU take as long as one after the
// other, so a started round counts whole. The constants come from timing every
// tile with 1 to 16 ranges on one MI355X:
//   row-major B: 40 shapes (M 32 to 5905, K 64 to 31744); the tile and ranges of
//     least time by the model were the fastest or within 8% of it on 38 of them.
//     M x N x K in us (calls for one output, operands from HBM): 2000 x 4096 x 14336
//     208 on 256 x 256 in two ranges, 247 on 128 x 128 in one; 161 x 2656 x 10624
//     32.5 on 64 x 128 in four (37.0 in three, 42.3 in five), 33.3 on 128 x 128 in
//     six; transposed 4096 x 14336 x 128 34.3 on 128 x 128, 42.4 on 256 x 256.
//   gated: 27 shapes (M 70 to 8192, K 320 to 8192); within 8% on 26. 259 x 4384 x
//     6592 38.9 on 128 x 256 in four ranges, 38.3 on 128 x 128 in two; 509 x 14336 x
//     4096 59.0 on 128 x 256, 64.7 on 128 x 128; 1536 x 1984 x 512 7.6 on 128 x 128,
//     10.3 on 128 x 256. The 256 x 256 tile's constants from 156 large ones (80 to
//     2100 GFLOP, M from 512, both types), every tile timed for 12 ms at a stretch,
//     as a training step's products run: at the clock that the power limit leaves it,
//     which is higher for the larger tile. The choice is 0.1% above the best of the
//     three largest tiles on average there, 3.2% at worst, and 0.1% and 1.8% on 56
//     others. 8192 x 28672 x 4096 1359 on 256 x 256, 1375 on 128 x 256, 1588 on 128 x
//     128; 6385 x 12384 x 8000 973, 1040; 7292 x 21472 x 512 169, 148.
struct TileTime { int tm, tn; double step, ends, join; };
constexpr TileTime kRowsTimes[] = {{256, 256, 1.21, 9.5, 3.2}, {128, 256, 0.99, 5.6, 2.1}, {128, 128, 0.60, 1.65, 1.25},
                                   {64, 128, 0.32, 2.15, 0.7}};
constexpr TileTime kGatedTimes[] = {{256, 256, 1.02, 15.4, 0}, {128, 256, 0.56, 6.0, 3.0}, {128, 128, 0.60, 1.25, 1.35},
                                    {64, 128, 0.35, 0.73, 1.0}};
double tile_us(const TileTime& t, int64_t M, int64_t N, int64_t Kb, int64_t ks, double speed = 1.0) {
  const double fill = (double)(((M + t.tm - 1) / t.tm) * ((N + t.tn - 1) / t.tn) * ks) / 256;
  const double rounds = fill <= 4 ? std::ceil(fill) : fill + 0.5;
  return 3.5 + rounds * ((double)Kb / 128 / ks * t.step * speed + t.ends) + (ks > 1 ? ks * t.join : 0);
}
// The tile and K ranges of least time, and that time; below 0 if no tile fits.
// inside: tiles no larger than the matrix.
double choose_tile_us(const TileTime (&times)[4], int64_t M, int64_t N, int64_t Kb, bool inside, Plan* p) {
  double best = -1;
  for (const TileTime& t : times) {
    if (inside && (t.tm > M || t.tn > N)) continue;
    const int64_t n = ((M + t.tm - 1) / t.tm) * ((N + t.tn - 1) / t.tn), kt = Kb / 128;
    for (int64_t ks = 1; ks <= 16; ++ks) {
      if (ks > 1 && (t.join == 0 || kt / ks < 4 || n * ks > 1024)) break;
      const double us = tile_us(t, M, N, Kb, ks);
      if (best >= 0 && us >= best) continue;
      best = us;
      *p = Plan();
      p->kernel = GP_KERNEL_TILE;
      p->tm = t.tm;
      p->tn = t.tn;
      p->tkb = 128;
      p->ks = (int)ks;
      p->Kb = Kb;
    }
  }
  return best;
}

// ---- gated product ----
struct GatedPlan {
  bool small = false;   // gated_small_kernel, else the tile kernel
  GatedSmall variant;
  int64_t ks = 1, tiles = 0, bytes = 0;   // small kernel: K ranges, workgroups of one, workspace
  Plan tile;
};

// The weights' K axis in whole 128-byte K tiles: 259 x 6560 x 2192 ran on 64-byte
// ones (K 6560 is 102.5 larger tiles) in 82 us, on 103 filled up tiles in 25.
int64_t whole_k(int64_t H) { return (H + 63) / 64 * 64; }

int check_gated(int dtype, int64_t M, int64_t F, int64_t H) {
  if (M <= 0 || F <= 0 || H <= 0) return GP_EINVAL;
  if (!half_type(dtype)) return GP_EDTYPE;
  if (M >= kMaxBytes || F >= kMaxBytes / 2 || H >= kMaxBytes) return GP_ESHAPE;
  if (F % 16 || H % 32) return GP_ESHAPE;
  if (!fits(M, 2 * H) || !fits(2 * F, 2 * whole_k(H)) || !fits(M, 4 * F)) return GP_ESHAPE;
  return GP_OK;
}

// Up to 64 rows, and above where no tile fits into [M][2F], the small gated
// kernel; otherwise a tile.
// Variants of the small kernel, F x H of 14336 x 4096 (896 pairs of column
// blocks), 7184 x 4096 (449) and 4096 x 4096 (256) unless named, us on one
// MI355X: up to 16 rows single pairs on 8 waves (1 x 7168 x 2048 10.8, pairs by
// two 11.4); 32 rows two pairs on 4 waves from 512 pairs on, 39.2 against 45.2
// on single ones, below single ones (256 pairs 15.0 against 21.2); 48 rows two
// pairs on 4 waves 42.9 (on 8 waves 46.0), below 512 pairs on 8 waves (37 rows,
// 449 pairs: 26.2, on 4 waves 27.4, single 27.9), below 384 single ones (18.4
// against 23.5); 64 rows four pairs 45.0 (two 49.1), below 768 two (7168 x 2048
// 16.5, single 17.8), below 384 single (20.4 against 24.9).
int plan_gated(int dtype, int64_t M, int64_t F, int64_t H, GatedPlan* p) {
  const int r = check_gated(dtype, M, F, H);
  if (r) return r;
  p->small = M <= 64;
  if (!p->small) p->small = choose_tile_us(kGatedTimes, M, 2 * F, 2 * whole_k(H), true, &p->tile) < 0;
  if (p->small) {
    GatedSmall& v = p->variant;
    const int64_t pairs = F / 16;
    v.xl = M == 1 ? 0 : M <= 8 ? 1 : M <= 16 ? 2 : M <= 32 ? 4 : M <= 48 ? 6 : 8;
    v.s = v.xl <= 2 || (v.xl == 4 && pairs < 512) ? 2 : 1;
    v.pairs = v.xl <= 2 ? 1 : v.xl == 4 ? (pairs >= 512 ? 2 : 1) : v.xl == 8 && pairs >= 768 ? 4 : pairs >= 384 ? 2 : 1;
    v.waves = v.xl <= 2 || (v.xl == 6 && v.pairs == 2 && pairs < 512) ? 8 : 4;
    const int64_t rows = v.xl == 0 ? 1 : 8 * v.xl;
    p->tiles = ((pairs + v.pairs - 1) / v.pairs) * ((M + rows - 1) / rows);
    if (p->tiles >= (int64_t)1 << 22) return GP_ESHAPE;   // threads of a grid
    const double step_us = v.xl <= 2 ? 0.5 : v.xl == 4 ? 0.35 : 0.65;
    p->ks = split_small((double)whole_k(H) / 64 / v.waves, step_us, p->tiles);
    if (p->ks > 1) p->bytes = kCounterBytes + p->tiles * p->ks * ((rows + 15) / 16 * v.pairs * 2048);
  } else {
    p->bytes = plan_workspace(p->tile, M, 2 * F);
  }
  return GP_OK;
}

// ---- backward pass of a linear layer C[M][N] = A[M][K] B[N][K]^T ----
// da = dc b: K axis N (gated: padded, since the call makes dc).
// db = dc^T a: K axis M, padded with zeros.
// Either runs on the tile kernel's row-major form: da reads b as it is; db is
// computed as (a^T dc)^T, which reads dc as it is, from a transposed copy of a
// (the smaller operand), and is stored transposed. Or on the preshuffled kernels,
// from copies laid out for them: b^T for da, dc^T and a^T for db. The copies cost
// bandwidth, the row-major products up to 14% of the matrix rate, so that the
// copies pay off with many rows; which one, plan_rows estimates. Gated backward M
// x F x H in us, row-major against copies: 130 x 2064 x 2048 22, 34; 512 x 4096 x
// 4096 100, 112; 2000 x 7168 x 4096 452, 483; 4096 x 11008 x 4096 1322, 1245; 8192 x
// 14336 x 4096 3229, 3039 (copies and the pointwise pass that also writes dc^T:
// 458 of these; the matrix unit is busy 88% of the products' cycles at the 1.65
// GHz that the power limit leaves).
struct BackwardPlan {
  Plan da, db;
  bool da_rows = false, db_rows = false, pair = false;   // pair: both in one launch
  int64_t Mp = 0, Np = 0;
  // workspace: counters and partial sums of the two products (the same ones after
  // each other; in a pair db's after da's), then the copies
  int64_t parts = 0, db_part = 0, off_bt = 0, off_at = 0, off_ct = 0, off_d = 0, bytes = 0;
};

int64_t align256(int64_t v) { return (v + 255) & ~(int64_t)255; }

// A K axis that the call itself lays out, filled up with zeros: to whole
// 128-byte K tiles, and for long ones, where the planner may split K across
// workgroups, so that it divides into several ranges; at most 1/16 more work.
// Measured: db of 2000 x 14336 x 4096 (K 2000) 241 us on the 64-byte K tiles of
// 2016, 222 us on the 128-byte tiles of 2048; da of 130 x 4128 x 2048 (K 4128)
// 46.8 us unsplit, 15 us on 4352 split in four.
int64_t pad_k(int64_t k) {
  const int64_t unit = k >= 16384 ? 1024 : k >= 4096 ? 256 : 64;
  return (k + unit - 1) / unit * unit;
}

// Tile and K ranges of the row-major form, where it is expected to take less
// time than the preshuffled plan `other` (null: none) with `copied` bytes of
// copies at the card's 4.9 TB/s; else false. On preshuffled operands a step takes
// about 0.85 of the row-major one. Always the row-major form where the planner
// answers with a small-M kernel or a tile outside kRowsTimes: of 32 such products
// (M 1 to 2821) da took 0.20 to 0.92 of the time that it takes from copies, db 0.58
// to 1.02 (a as it is: 10 x 10304 x 4480 25.0 us, from copies 117; 29 x 224 x 1728 db
// 11.9, 11.8).
bool plan_rows(int64_t M, int64_t N, int64_t Kb, const Plan* other, double copied, Plan* p, double* took) {
  const double us = *took = choose_tile_us(kRowsTimes, M, N, Kb, false, p);
  if (!other || other->kernel != GP_KERNEL_TILE) return true;
  for (const TileTime& t : kRowsTimes)
    if (t.tm == other->tm && t.tn == other->tn) return us <= tile_us(t, M, N, Kb, other->ks, 0.85) + copied / 4.9e6;
  return true;
}

// Both products in one launch, on 64 x 128 tiles: a [Ma][Na] over Ka K tiles, b
// likewise. The workgroups share the CUs, two on each, so the time is that of all
// their work, or of the longest, slowed by what runs beside it:
//   3.5 + max(sum of (K tiles * 0.27 + 0.3) / 256, 1.4 * longest + 0.5) + joins (us)
// taken where it is 5% below the two products' times (it also saves a launch). On
// 25 shapes timed with every pair of ranges the choice was 3% above the best of
// both on average, 17% at worst. Gated calls of M x F x H, one launch of the products
// against two: 130 x 2064 x 2048 21.8, 27.7; 1116 x 672 x 480 17.7, 25.9; 57 x 3392 x
// 2080 22.3, 27.2; 606 x 4896 x 448 33.5, 41.2; 682 x 5808 x 608 53.1, 57.0.
bool plan_pair(int64_t Ma, int64_t Na, int64_t Ka, int64_t Mb, int64_t Nb, int64_t Kb, double apart, Plan* a, Plan* b) {
  const int64_t ta = ((Ma + 63) / 64) * ((Na + 127) / 128), tb = ((Mb + 63) / 64) * ((Nb + 127) / 128);
  if (ta + tb > 2304) return false;   // 512 x 4096 x 4096 (4352 tiles) 89 us, apart on larger tiles 80
  double best = 0.95 * apart;
  bool found = false;
  for (int64_t x = 1; x <= 16 && (x == 1 || (Ka / x >= 4 && ta * x <= 1024)); ++x)
    for (int64_t y = 1; y <= 16 && (y == 1 || (Kb / y >= 4 && tb * y <= 1024)); ++y) {
      const double wa = 0.27 * (double)Ka / x + 0.3, wb = 0.27 * (double)Kb / y + 0.3;
      const double us = 3.5 + std::max((ta * x * wa + tb * y * wb) / 256, 1.4 * std::max(wa, wb) + 0.5) +
                        (double)(x > 1 ? x : 0) + (double)(y > 1 ? y : 0);
      if (us >= best) continue;
      best = us;
      found = true;
      for (Plan* p : {a, b}) {
        *p = Plan();
        p->kernel = GP_KERNEL_TILE;
        p->tm = 64;
        p->tn = 128;
        p->tkb = 128;
      }
      a->ks = (int)x;
      a->Kb = Ka * 128;
      b->ks = (int)y;
      b->Kb = Kb * 128;
    }
  return found;
}

// gated: dc itself is made by the call ([M][Np] in the workspace).
int make_backward_plan(int dtype, int64_t M, int64_t N, int64_t K, bool want_da, bool want_db, bool gated, BackwardPlan* p) {
  if (M <= 0 || N <= 0 || K <= 0) return GP_EINVAL;
  if (!half_type(dtype)) return GP_EDTYPE;
  if (M >= kMaxBytes / 4 || N >= kMaxBytes || K >= kMaxBytes) return GP_ESHAPE;
  if (N % 32 || K % 32) return GP_ESHAPE;
  p->Mp = pad_k(M);
  p->Np = gated ? pad_k(N) : N;
  if (!fits(p->Mp, 2 * K) || !fits(p->Np, 2 * K) || !fits(p->Mp, 2 * p->Np)) return GP_ESHAPE;
  // both products are planned whichever are wanted, so that an output has the same
  // bits with and without the other. One output alone then runs on the pair's tile:
  // on 31 sizes against the tile that the model has for it alone (with the pair's
  // ranges) 24 took the same time within 2%, 4 up to 8% less, 3 more: da of 1500 x
  // 5984 x 800 40.5 us against 34.9, db of 1319 x 5280 x 704 21.1 against 19.1.
  Plan copies, copies_b;   // (one each: the planner sets what differs from a new Plan)
  double us_a = 0, us_b = 0;
  int r = plan_gemm(dtype, M, K, p->Np, &copies);
  p->da_rows = plan_rows(M, K, 2 * whole_k(p->Np), r ? nullptr : &copies, 4.0 * p->Np * K, &p->da, &us_a);
  if (!p->da_rows) p->da = copies;
  r = plan_gemm(dtype, N, K, p->Mp, &copies_b);
  p->db_rows = plan_rows(K, N, 2 * p->Mp, r ? nullptr : &copies_b, (gated ? 2.0 : 4.0) * p->Mp * N, &p->db, &us_b);
  if (!p->db_rows) p->db = copies_b;
  p->pair = p->da_rows && p->db_rows &&
            plan_pair(M, K, whole_k(p->Np) / 64, K, N, p->Mp / 64, us_a + us_b, &p->da, &p->db) && want_da && want_db;
  const int64_t part_a = want_da ? plan_workspace(p->da, M, K) : 0;
  const int64_t part_b = want_db ? (p->db_rows ? plan_workspace(p->db, K, N) : plan_workspace(p->db, N, K)) : 0;
  int64_t parts = std::max(part_a, part_b);
  if (p->pair && parts > 0) {
    p->db_part = std::max(part_a, kCounterBytes);
    parts = p->db_part + part_b;   // (which counts the counters once more)
  }
  int64_t at = p->parts = align256(parts);
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += align256(bytes);
    return here;
  };
  p->off_bt = take(want_da && !p->da_rows ? p->Np * K * 2 : 0);
  p->off_at = take(want_db ? p->Mp * K * 2 : 0);
  p->off_ct = take(want_db && !p->db_rows ? p->Mp * N * 2 : 0);
  p->off_d = take(gated && (want_da || p->db_rows) ? M * p->Np * 2 : 0);
  p->bytes = std::max<int64_t>(at, 256);   // never none: one rule for every caller
  return GP_OK;
}

// A plan depends on these numbers alone and takes 3 to 6 us to make, as long as a
// launch; a training loop asks for a few of them over and over. Kept per thread,
// the latest of each slot.
int plan_backward(int dtype, int64_t M, int64_t N, int64_t K, bool want_da, bool want_db, bool gated, BackwardPlan* p) {
  struct Slot {
    int64_t key[4] = {-1, 0, 0, 0};
    BackwardPlan plan;
  };
  static thread_local Slot slots[32];
  const int64_t key[4] = {(int64_t)dtype * 8 + want_da * 4 + want_db * 2 + gated, M, N, K};
  uint64_t h = 0;
  for (int64_t k : key) h = (h ^ (uint64_t)k) * 0x9E3779B97F4A7C15ull;
  Slot& s = slots[h >> 59];
  if (key[0] >= 0 && std::equal(key, key + 4, s.key)) {
    *p = s.plan;
    return GP_OK;
  }
  const int r = make_backward_plan(dtype, M, N, K, want_da, want_db, gated, p);
  if (r == GP_OK) {
    std::copy(key, key + 4, s.key);
    s.plan = *p;
  }
  return r;
}

uint32_t tiles64(int64_t R, int64_t C) { return (uint32_t)(((R + 63) / 64) * ((C + 63) / 64)); }

// a [M][lda] (K fast) times b [rows][N] row-major, K filled up to p.Kb bytes with
// zeros past lda and rows; c [M][N], or (transposed form) [N][M].
TileArgs rows_args(const Plan& p, const void* a, int64_t lda, const void* b, void* c, int64_t M, int64_t N,
                   int64_t rows, int64_t ldb, char* counters, char* part) {
  TileArgs g;
  g.a = (const char*)a;
  g.b = (const char*)b;
  g.sa = g.sb = nullptr;
  g.bias = nullptr;
  g.c = (char*)c;
  g.M = (uint32_t)M;
  g.N = (uint32_t)N;
  g.Kb = (uint32_t)p.Kb;
  g.ka = (uint32_t)(2 * lda);
  g.tiles_m = (uint32_t)((M + p.tm - 1) / p.tm);
  g.tiles_n = (uint32_t)((N + p.tn - 1) / p.tn);
  g.xcd = 1;
  g.act = ACT_NONE;
  g.gate = g.up = nullptr;
  g.kb_rows = (uint32_t)rows;
  g.ldb = (uint32_t)(2 * ldb);
  g.ksplit = (uint32_t)p.ks;
  g.cnt = p.ks > 1 ? (uint32_t*)counters : nullptr;
  g.part = p.ks > 1 ? part : nullptr;
  return g;
}

// Launches, in order, what has to run once the pointers are valid. dc: the
// output gradient, rows of ldc elements; gate: the pointwise backward that makes
// it first (else null). Stops at the first launch that fails.
int run_backward(int dtype, const BackwardPlan& p, const GateGradArgs* gate, const void* dc, const void* a,
                 const void* b, void* da, void* db, int64_t M, int64_t N, int64_t K, char* ws, hipStream_t s) {
  const int64_t ldc = gate ? p.Np : N;
  PrepArgs t = {};
  uint64_t blocks = 0;
  if (gate) {
    t.gate = *gate;
    blocks = t.gate.blocks = tiles64(p.Mp, t.gate.F);
  }
  int jobs = 0;
  auto copy = [&](const void* src, int64_t off, int64_t R, int64_t C, int64_t Kp, bool preshuffled) {
    CopyJob& j = t.copy[jobs++];
    j.src = (const char*)src;
    j.dst = ws + off;
    j.R = (uint32_t)R;
    j.C = (uint32_t)C;
    j.Kp = (uint32_t)Kp;
    j.tiles_c = (uint32_t)((C + 63) / 64);
    j.blocks = tiles64(Kp, C);
    j.preshuffled = preshuffled;
    blocks += j.blocks;
  };
  if (da && !p.da_rows) copy(b, p.off_bt, N, K, p.Np, true);
  if (db) copy(a, p.off_at, M, K, p.Mp, !p.db_rows);
  if (db && !p.db_rows && !gate) copy(dc, p.off_ct, M, N, p.Mp, false);
  if (p.parts > 0) {
    // arrival counters of the K splits: cleared here, so that the workspace
    // needs no state from earlier calls
    t.cnt = (uint32_t*)ws;
    t.ncnt = (uint32_t)(kCounterBytes / 4);
    blocks = std::max<uint64_t>(blocks, 16);
  }
  int r;
  if (blocks > 0) {
    forget_hip_error();
    if (dtype == GP_BF16) hipLaunchKernelGGL((prep_kernel<DT_BF16>), dim3((uint32_t)blocks), dim3(256), 0, s, t);
    else hipLaunchKernelGGL((prep_kernel<DT_F16>), dim3((uint32_t)blocks), dim3(256), 0, s, t);
    if ((r = report_hip(hipGetLastError(), "kernel launch"))) return r;
  }
  const bool bf16 = dtype == GP_BF16;
  TileArgs ra = {}, rb = {};
  if (da && p.da_rows) ra = rows_args(p.da, dc, ldc, b, da, M, K, N, K, ws, ws + kCounterBytes);
  if (db && p.db_rows) rb = rows_args(p.db, ws + p.off_at, p.Mp, dc, db, K, N, M, ldc, ws, ws + kCounterBytes);
  if (p.pair) {
    // db's counters follow da's, its partial sums da's
    if (p.db.ks > 1) {
      rb.cnt = (uint32_t*)ws + ra.tiles_m * ra.tiles_n;
      rb.part = ws + p.db_part;
    }
    forget_hip_error();
    return report_hip(bf16 ? launch_pair_bf16(ra, rb, s) : launch_pair_f16(ra, rb, s), "kernel launch");
  }
  auto launch_rows = [&](const Plan& plan, const TileArgs& g, bool t) {
    forget_hip_error();
    auto* launch = bf16 ? (t ? launch_rows_t_bf16 : launch_rows_bf16) : (t ? launch_rows_t_f16 : launch_rows_f16);
    return report_hip(launch(plan.tm, plan.tn, g, s), "kernel launch");
  };
  if (da) {
    r = p.da_rows ? launch_rows(p.da, ra, false)
                  : launch_gemm(dtype, p.da, dc, ws + p.off_bt, da, M, K, ws, s);
    if (r) return r;
  }
  if (db) {
    r = p.db_rows ? launch_rows(p.db, rb, true)
                  : launch_gemm(dtype, p.db, ws + p.off_ct, ws + p.off_at, db, N, K, ws, s);
    if (r) return r;
  }
  return GP_OK;
}

int plan_gated_backward(int dtype, int64_t M, int64_t F, int64_t H, bool dx, bool dw, BackwardPlan* p) {
  const int r = check_gated(dtype, M, F, H);
  if (r) return r;
  return plan_backward(dtype, M, 2 * F, H, dx, dw, true, p);
}

}  // namespace
}  // namespace gp

using namespace gp;

extern "C" {

int gemm_gated_preshuffle(const void* w, void* w_shuf, int64_t F, int64_t H, int dtype, void* stream) {
  if (!w || !w_shuf || !is_aligned16(w) || !is_aligned16(w_shuf)) return GP_EINVAL;
  int r = check_gated(dtype, 1, F, H);
  if (r) return r;
  const int64_t bytes = 4 * F * whole_k(H);
  const char *wb = (const char*)w, *sb = (const char*)w_shuf;
  if (sb < wb + 4 * F * H && wb < sb + bytes) return GP_EINVAL;   // overlap
  if ((r = require_gfx950())) return r;
  const uint32_t chunks = (uint32_t)(bytes / 16);
  forget_hip_error();
  hipLaunchKernelGGL(preshuffle_gated_kernel, dim3((chunks + 255) / 256), dim3(256), 0, (hipStream_t)stream, wb,
                     (char*)w_shuf, (uint32_t)(whole_k(H) / 32), (uint32_t)(2 * H), (uint32_t)F, chunks);
  return report_hip(hipGetLastError(), "kernel launch");
}

int gemm_gated_workspace_size(int dtype, int64_t M, int64_t F, int64_t H, size_t* bytes) {
  if (!bytes) return GP_EINVAL;
  GatedPlan p;
  const int r = plan_gated(dtype, M, F, H, &p);
  if (r) return r;
  *bytes = (size_t)p.bytes;
  return GP_OK;
}

int gemm_gated_plan(int dtype, int64_t M, int64_t F, int64_t H, gemm_plan_info* out) {
  if (!out) return GP_EINVAL;
  GatedPlan p;
  const int r = plan_gated(dtype, M, F, H, &p);
  if (r) return r;
  *out = gemm_plan_info();
  const int64_t rows = p.variant.xl == 0 ? 1 : 8 * p.variant.xl;
  out->kernel = p.small ? GP_KERNEL_SPLITK : GP_KERNEL_TILE;
  out->tile_m = p.small ? (int)rows : p.tile.tm;
  out->tile_n = p.small ? 32 * p.variant.pairs : p.tile.tn;
  out->tile_k = p.small ? 64 * p.variant.s : 64;
  out->waves = p.small ? p.variant.waves : tile_waves(p.tile.tm, p.tile.tn);
  out->threads = 64 * out->waves;
  out->ksplit = p.small ? (int)p.ks : p.tile.ks;
  out->grid = out->ksplit * (p.small ? p.tiles : (M + p.tile.tm - 1) / p.tile.tm * ((2 * F + p.tile.tn - 1) / p.tile.tn));
  out->mfma = 16;
  out->workspace_bytes = p.bytes;
  return GP_OK;
}

int gemm_gated(int dtype, const void* x, const void* w_shuf, int act, void* h, void* gate, void* up, int64_t M,
               int64_t F, int64_t H, void* workspace, size_t workspace_bytes, void* stream) {
  if (!x || !w_shuf || !h || !is_aligned16(x) || !is_aligned16(w_shuf) || !is_aligned16(h)) return GP_EINVAL;
  if (!gate != !up || !is_aligned16(gate) || !is_aligned16(up)) return GP_EINVAL;
  if (act < GP_ACT_NONE || act > GP_ACT_GELU) return GP_EINVAL;
  GatedPlan p;
  int r = plan_gated(dtype, M, F, H, &p);
  if (r) return r;
  if (p.bytes > 0) {
    if (!workspace || (int64_t)workspace_bytes < p.bytes) return GP_EWORKSPACE;
    if (!is_aligned16(workspace)) return GP_EINVAL;
  }
  if ((r = require_gfx950())) return r;
  const hipStream_t s = (hipStream_t)stream;
  forget_hip_error();
  hipError_t e;
  if (p.small) {
    GatedArgs t;
    t.a = (const char*)x;
    t.b = (const char*)w_shuf;
    t.c = (char*)h;
    t.gate = (char*)gate;
    t.up = (char*)up;
    t.M = (uint32_t)M;
    t.F = (uint32_t)F;
    t.Ka = (uint32_t)(2 * H);
    t.Kb = (uint32_t)(2 * whole_k(H));
    t.act = act;
    t.ksplit = (uint32_t)p.ks;
    t.cnt = p.ks > 1 ? (uint32_t*)workspace : nullptr;
    t.part = p.ks > 1 ? (char*)workspace + kCounterBytes : nullptr;
    e = dtype == GP_BF16 ? launch_gated_small_bf16(p.variant, t, s) : launch_gated_small_f16(p.variant, t, s);
  } else {
    TileArgs t;
    t.a = (const char*)x;
    t.b = (const char*)w_shuf;
    t.sa = t.sb = nullptr;
    t.bias = nullptr;
    t.c = (char*)h;
    t.M = (uint32_t)M;
    t.N = (uint32_t)(2 * F);
    t.Kb = (uint32_t)(2 * whole_k(H));
    t.ka = (uint32_t)(2 * H);
    t.tiles_m = (uint32_t)((M + p.tile.tm - 1) / p.tile.tm);
    t.tiles_n = (uint32_t)((2 * F + p.tile.tn - 1) / p.tile.tn);
    t.xcd = 1;
    t.act = act;
    t.gate = (char*)gate;
    t.up = (char*)up;
    t.kb_rows = t.ldb = 0;
    t.ksplit = (uint32_t)p.tile.ks;
    t.cnt = p.tile.ks > 1 ? (uint32_t*)workspace : nullptr;
    t.part = p.tile.ks > 1 ? (char*)workspace + kCounterBytes : nullptr;
    e = dtype == GP_BF16 ? launch_gated_tile_bf16(p.tile.tm, p.tile.tn, t, s)
                         : launch_gated_tile_f16(p.tile.tm, p.tile.tn, t, s);
  }
  return report_hip(e, "kernel launch");
}

int gemm_backward_workspace_size(int dtype, int64_t M, int64_t N, int64_t K, int want_da, int want_db, size_t* bytes) {
  if (!bytes || (!want_da && !want_db)) return GP_EINVAL;
  BackwardPlan p;
  const int r = plan_backward(dtype, M, N, K, want_da != 0, want_db != 0, false, &p);
  if (r) return r;
  *bytes = (size_t)p.bytes;
  return GP_OK;
}

int gemm_backward_plan(int dtype, int64_t M, int64_t N, int64_t K, int want_da, int want_db, int gated,
                       gemm_plan_info* da, gemm_plan_info* db) {
  if (!da || !db || (!want_da && !want_db)) return GP_EINVAL;
  BackwardPlan p;
  const int r = gated ? plan_gated_backward(dtype, M, N, K, want_da != 0, want_db != 0, &p)
                      : plan_backward(dtype, M, N, K, want_da != 0, want_db != 0, false, &p);
  if (r) return r;
  *da = *db = gemm_plan_info();
  auto fill = [&](const Plan& q, bool rows, int64_t m, int64_t n, int64_t k, gemm_plan_info* out) {
    if (!rows) report_plan(dtype, m, n, k, q, out);
    else {
      out->kernel = p.pair ? GP_KERNEL_PAIR : GP_KERNEL_ROWS;
      out->tile_m = q.tm;
      out->tile_n = q.tn;
      out->tile_k = 64;
      out->waves = tile_waves(q.tm, q.tn);
      out->threads = 64 * out->waves;
      out->ksplit = q.ks;
      out->grid = (m + q.tm - 1) / q.tm * ((n + q.tn - 1) / q.tn) * q.ks;
      out->mfma = 16;
    }
    out->workspace_bytes = p.bytes;
  };
  const int64_t rows = gated ? 2 * N : N;
  if (want_da) fill(p.da, p.da_rows, M, K, p.Np, da);
  if (want_db) fill(p.db, p.db_rows, p.db_rows ? K : rows, p.db_rows ? rows : K, p.Mp, db);
  return GP_OK;
}

int gemm_backward(int dtype, const void* dc, const void* a, const void* b, void* da, void* db, int64_t M, int64_t N,
                  int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dc || !is_aligned16(dc) || (!da && !db)) return GP_EINVAL;
  if ((da && !b) || (db && !a)) return GP_EINVAL;
  if (!is_aligned16(a) || !is_aligned16(b) || !is_aligned16(da) || !is_aligned16(db)) return GP_EINVAL;
  BackwardPlan p;
  int r = plan_backward(dtype, M, N, K, da != nullptr, db != nullptr, false, &p);
  if (r) return r;
  if (!workspace || (int64_t)workspace_bytes < p.bytes) return GP_EWORKSPACE;
  if (!is_aligned16(workspace)) return GP_EINVAL;
  if ((r = require_gfx950())) return r;
  return run_backward(dtype, p, nullptr, dc, a, b, da, db, M, N, K, (char*)workspace, (hipStream_t)stream);
}

int gemm_gated_backward_workspace_size(int dtype, int64_t M, int64_t F, int64_t H, int want_dx, int want_dw,
                                       size_t* bytes) {
  if (!bytes || (!want_dx && !want_dw)) return GP_EINVAL;
  BackwardPlan p;
  const int r = plan_gated_backward(dtype, M, F, H, want_dx != 0, want_dw != 0, &p);
  if (r) return r;
  *bytes = (size_t)p.bytes;
  return GP_OK;
}

int gemm_gated_backward(int dtype, const void* dh, const void* gate, const void* up, const void* x, const void* w,
                        int act, void* dx, void* dw, int64_t M, int64_t F, int64_t H, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!dh || !gate || !up || (!dx && !dw)) return GP_EINVAL;
  if ((dx && !w) || (dw && !x)) return GP_EINVAL;
  if (!is_aligned16(dh) || !is_aligned16(gate) || !is_aligned16(up) || !is_aligned16(x) || !is_aligned16(w) ||
      !is_aligned16(dx) || !is_aligned16(dw))
    return GP_EINVAL;
  if (act < GP_ACT_NONE || act > GP_ACT_GELU) return GP_EINVAL;
  BackwardPlan p;
  int r = plan_gated_backward(dtype, M, F, H, dx != nullptr, dw != nullptr, &p);
  if (r) return r;
  if (!workspace || (int64_t)workspace_bytes < p.bytes) return GP_EWORKSPACE;
  if (!is_aligned16(workspace)) return GP_EINVAL;
  if ((r = require_gfx950())) return r;
  char* ws = (char*)workspace;
  GateGradArgs t;
  t.dh = (const char*)dh;
  t.gate = (const char*)gate;
  t.up = (const char*)up;
  t.d = dx || p.db_rows ? ws + p.off_d : nullptr;
  t.dt = dw && !p.db_rows ? ws + p.off_ct : nullptr;
  t.M = (uint32_t)M;
  t.F = (uint32_t)F;
  t.Mp = (uint32_t)p.Mp;
  t.Np = (uint32_t)p.Np;
  t.tiles_c = (uint32_t)((F + 63) / 64);
  t.act = act;
  return run_backward(dtype, p, &t, ws + p.off_d, x, w, dx, dw, M, 2 * F, H, ws, (hipStream_t)stream);
}

}  // extern "C"
