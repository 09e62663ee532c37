// Launch tables of the gated product (BF16 and FP16).
#pragma once

#include "gated_small.hpp"
#include "gemm_tile.hpp"

namespace gp {

// A variant of gated_small_kernel: x loads (0: one row, else rows / 8), column
// pairs, waves, 64-element K chunks per group.
struct GatedSmall {
  int xl = 0, pairs = 1, waves = 8, s = 2;
};

// Each returns hipErrorInvalidValue if the variant is not compiled.
hipError_t launch_gated_tile_bf16(int tm, int tn, const TileArgs& a, hipStream_t s);
hipError_t launch_gated_tile_f16(int tm, int tn, const TileArgs& a, hipStream_t s);
hipError_t launch_gated_small_bf16(const GatedSmall& v, const GatedArgs& a, hipStream_t s);
hipError_t launch_gated_small_f16(const GatedSmall& v, const GatedArgs& a, hipStream_t s);

}  // namespace gp

#define GP_GATED_CASE(DT, TM, TN, KSV)                                                                         \
  if (tm == TM && tn == TN && (a.ksplit > 1) == KSV) {                                                         \
    hipLaunchKernelGGL((gemm_tile_kernel<DT, 16, TM, TN, 128, EPI_GATED, 3, false, 1, true, KSV>),             \
                       dim3(a.tiles_m * a.tiles_n * a.ksplit), dim3(64 * tile_waves(TM, TN)), 0, s, a);        \
    return hipGetLastError();                                                                                  \
  }
#define GP_GATED_SMALL_CASE(DT, XL, P, W, S)                                                                   \
  if (v.xl == XL && v.pairs == P && v.waves == W && v.s == S) {                                                \
    constexpr uint32_t rows = XL == 0 ? 1 : 8 * XL;                                                            \
    const dim3 grid(((a.F / 16 + P - 1) / P) * ((a.M + rows - 1) / rows) * a.ksplit);                          \
    hipLaunchKernelGGL((gated_small_kernel<DT, XL, P, W, S>), grid, dim3(W * 64), 0, s, a);                    \
    return hipGetLastError();                                                                                  \
  }
#define GP_DEFINE_GATED(NAME, DT)                                                                              \
  hipError_t launch_gated_tile_##NAME(int tm, int tn, const TileArgs& a, hipStream_t s) {                      \
    GP_TILE_GATED(GP_GATED_CASE, DT)                                                                           \
    return hipErrorInvalidValue;                                                                               \
  }                                                                                                            \
  hipError_t launch_gated_small_##NAME(const GatedSmall& v, const GatedArgs& a, hipStream_t s) {               \
    GP_GATED_SMALL_CASE(DT, 0, 1, 8, 2)                                                                        \
    GP_GATED_SMALL_CASE(DT, 1, 1, 8, 2)                                                                        \
    GP_GATED_SMALL_CASE(DT, 2, 1, 8, 2)                                                                        \
    GP_GATED_SMALL_CASE(DT, 4, 1, 4, 2)                                                                        \
    GP_GATED_SMALL_CASE(DT, 4, 2, 4, 1)                                                                        \
    GP_GATED_SMALL_CASE(DT, 6, 1, 4, 1)                                                                        \
    GP_GATED_SMALL_CASE(DT, 6, 2, 8, 1)                                                                        \
    GP_GATED_SMALL_CASE(DT, 6, 2, 4, 1)                                                                        \
    GP_GATED_SMALL_CASE(DT, 8, 1, 4, 1)                                                                        \
    GP_GATED_SMALL_CASE(DT, 8, 2, 4, 1)                                                                        \
    GP_GATED_SMALL_CASE(DT, 8, 4, 4, 1)                                                                        \
    return hipErrorInvalidValue;                                                                               \
  }
