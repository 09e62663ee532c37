// Launch tables of the linear layer with its epilogue (BF16 and FP16).
#pragma once

#include "ffn_small.hpp"
#include "gemm_tile.hpp"

namespace gp {

// A variant of ffn_small_kernel<linear>: x loads (0: one row, else rows / 8), column
// blocks, waves, 64-element K chunks per group.
struct LinearSmall {
  int xl = 0, blocks = 1, waves = 8, s = 2;
};

// Each returns hipErrorInvalidValue if the variant is not compiled.
hipError_t launch_linear_tile_bf16(int tm, int tn, const TileArgs& a, hipStream_t s);
hipError_t launch_linear_tile_f16(int tm, int tn, const TileArgs& a, hipStream_t s);
hipError_t launch_linear_small_bf16(const LinearSmall& v, const GatedArgs& a, hipStream_t s);
hipError_t launch_linear_small_f16(const LinearSmall& v, const GatedArgs& a, hipStream_t s);

}  // namespace gp

#define GP_LINEAR_CASE(DT, TM, TN, KSV)                                                                        \
  if (tm == TM && tn == TN && (a.ksplit > 1) == KSV) {                                                         \
    hipLaunchKernelGGL((gemm_tile_kernel<DT, 16, TM, TN, 128, EPI_LINEAR, 3, true, 1, true, KSV>),             \
                       dim3(a.tiles_m * a.tiles_n * a.ksplit), dim3(64 * tile_waves(TM, TN)), 0, s, a);        \
    return hipGetLastError();                                                                                  \
  }
#define GP_LINEAR_SMALL_CASE(DT, XL, NB, W, S)                                                                 \
  if (v.xl == XL && v.blocks == NB && v.waves == W && v.s == S) {                                              \
    constexpr uint32_t rows = XL == 0 ? 1 : 8 * XL;                                                            \
    const dim3 grid(((a.F / 16 + NB - 1) / NB) * ((a.M + rows - 1) / rows) * a.ksplit);                        \
    hipLaunchKernelGGL((ffn_small_kernel<DT, XL, NB, W, S, false>), grid, dim3(W * 64), 0, s, a);              \
    return hipGetLastError();                                                                                  \
  }
#define GP_DEFINE_LINEAR(NAME, DT)                                                                             \
  hipError_t launch_linear_tile_##NAME(int tm, int tn, const TileArgs& a, hipStream_t s) {                     \
    GP_TILE_LINEAR(GP_LINEAR_CASE, DT)                                                                         \
    return hipErrorInvalidValue;                                                                               \
  }                                                                                                            \
  hipError_t launch_linear_small_##NAME(const LinearSmall& v, const GatedArgs& a, hipStream_t s) {             \
    GP_SMALL_LINEAR(GP_LINEAR_SMALL_CASE, DT)                                                                  \
    return hipErrorInvalidValue;                                                                               \
  }
