// What the host sides of the library share: size limits, the GEMM planner and
// launcher, the device check and the HIP status kept for the caller.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gemm_preshuffle.h"
#include "gp_common.hpp"

namespace gp {

constexpr int64_t kMaxBytes = (int64_t)1 << 31;  // 32-bit buffer offsets

// rows * row_bytes < kMaxBytes, decided without forming the product (rows and
// row_bytes are positive; a product of two sizes near 2^62 would overflow)
inline bool fits(int64_t rows, int64_t row_bytes) { return row_bytes < kMaxBytes && rows <= (kMaxBytes - 1) / row_bytes; }

struct Plan {
  int kernel = 0;
  int ms = 16;                  // MFMA block (16 or 32)
  int pipe = 0;                 // 0 VGPR-staged A, 2 .. 6 LDS DMA stages
  int tm = 0, tn = 0, tkb = 0;  // tile and wide kernels (tkb in bytes)
  int kg = 1;                   // tile kernel: K groups of 4 waves
  int epi = EPI_DIRECT;
  int xcd = 1;
  int nb = 0, waves = 4, kch = 0, mb = 1;  // split-K kernel (mb: 16-row blocks per workgroup)
  int ks = 1;                   // tile kernel: K split across workgroups
  int sched = 1;                // tile kernel: 1 pinned hot-loop schedule, 2 the compiler's
  int64_t Kb = 0;
};

// Workspace of a K split across workgroups: a fixed area of arrival counters
// (4 bytes per tile, for up to kMaxSplitTiles tiles), then ks partial tiles of
// TM x TN 4-byte sums per tile. The counter area is the same for every
// shape, so a workspace whose counters are zero (as every call leaves them)
// can serve calls of any shape: a later call's counters never fall where an
// earlier call left partial sums.
constexpr int64_t kMaxSplitTiles = 16384;
constexpr int64_t kCounterBytes = kMaxSplitTiles * 4;

// Implemented beside the GEMM entry points (api.hip).
// The plan of gemm_ex_ws with no options (it may split K across workgroups),
// and the workspace bytes that plan needs (0: none).
int plan_gemm(int in_dtype, int64_t M, int64_t N, int64_t K, Plan* p);
int64_t plan_workspace(const Plan& p, int64_t M, int64_t N);
void report_plan(int in_dtype, int64_t M, int64_t N, int64_t K, const Plan& p, gemm_plan_info* out);
// Launch of a BF16 / FP16 plan, plain epilogue; pointers already validated.
int launch_gemm(int in_dtype, const Plan& p, const void* a, const void* b_shuf, void* c, int64_t M, int64_t N,
                void* ws, hipStream_t s);
// Records a HIP status and the call that returned it; the gp_status it maps to.
int report_hip(hipError_t e, const char* call);
// Clears HIP's per-thread last error (right before a launch).
void forget_hip_error();
// GP_OK on gfx950, else GP_EARCH or GP_EHIP.
int require_gfx950();

// K ranges of a small-M kernel whose waves run `steps` chunks of `step_us` each, on
// `tiles` workgroups: the ranges (one workgroup per CU and 16 at most) for which
// the chunks and the join, 0.8 us and 0.45 per range, take the least time. Measured
// on 22 shapes with 1 to 16 ranges: gated 1 x 368 x 6784 11.1 us unsplit, 7.5 in
// four, 11.5 in 16; 40 x 336 x 6720 21.2, 9.6 in six; 1 x 1024 x 2048 5.3, 6.1 in two.
inline int64_t split_small(double steps, double step_us, int64_t tiles) {
  double best = steps * step_us;
  int64_t ks = 1;
  for (int64_t k = 2; k <= 16 && tiles * k <= 256 && steps / (double)k >= 1; ++k) {
    const double us = steps * step_us / (double)k + 0.8 + 0.45 * (double)k;
    if (us < best) {
      best = us;
      ks = k;
    }
  }
  return ks;
}

inline bool is_aligned16(const void* ptr) { return ((uintptr_t)ptr & 15u) == 0; }

}  // namespace gp
