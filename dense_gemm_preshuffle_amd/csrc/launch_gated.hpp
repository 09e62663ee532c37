// Launch tables of the gated product (BF16 and FP16).
#pragma once

#include "gated_small.hpp"
#include "gemm_tile.hpp"

namespace gp {

// Each returns hipErrorInvalidValue if the variant is not compiled.
hipError_t launch_gated_tile_bf16(int tm, int tn, int tkb, int pipe, const TileArgs& a, hipStream_t s);
hipError_t launch_gated_tile_f16(int tm, int tn, int tkb, int pipe, const TileArgs& a, hipStream_t s);
hipError_t launch_gated_small_bf16(int mb, int waves, const GatedArgs& a, hipStream_t s);
hipError_t launch_gated_small_f16(int mb, int waves, const GatedArgs& a, hipStream_t s);

}  // namespace gp

#define GP_GATED_CASE_IMPL(DT, MS, TM, TN, TKB, PIPE, KSV)                                                     \
  if (tm == TM && tn == TN && tkb == TKB && pipe == PIPE && (a.ksplit > 1) == KSV) {                           \
    hipLaunchKernelGGL((gemm_tile_kernel<DT, MS, TM, TN, TKB, EPI_GATED, PIPE, false, 1, true, KSV>),          \
                       dim3(a.tiles_m * a.tiles_n * a.ksplit), dim3(64 * tile_waves(TM, TN)), 0, s, a);        \
    return hipGetLastError();                                                                                  \
  }
#define GP_GATED_CASE(DT, MS, TM, TN, TKB, PIPE) GP_GATED_CASE_IMPL(DT, MS, TM, TN, TKB, PIPE, false)
#define GP_GATED_CASE_KSPLIT(DT, MS, TM, TN, TKB, PIPE) GP_GATED_CASE_IMPL(DT, MS, TM, TN, TKB, PIPE, true)
#define GP_GATED_SMALL_CASE(DT, MB, P, W, S)                                                                   \
  if (mb == MB && waves == W) {                                                                                \
    const dim3 grid(((a.F / 16 + P - 1) / P) * ((a.M + 16 * MB - 1) / (16 * MB)));                              \
    hipLaunchKernelGGL((gated_small_kernel<DT, MB, P, W, S>), grid, dim3(W * 64), 0, s, a);                    \
    return hipGetLastError();                                                                                  \
  }
// (rows / 16, column pairs, waves, 64-byte K blocks per chunk)
#define GP_DEFINE_GATED(NAME, DT, TILES, KSPLIT)                                                               \
  hipError_t launch_gated_tile_##NAME(int tm, int tn, int tkb, int pipe, const TileArgs& a, hipStream_t s) {   \
    TILES(GP_GATED_CASE)                                                                                       \
    KSPLIT(GP_GATED_CASE_KSPLIT)                                                                               \
    return hipErrorInvalidValue;                                                                               \
  }                                                                                                            \
  hipError_t launch_gated_small_##NAME(int mb, int waves, const GatedArgs& a, hipStream_t s) {                 \
    GP_GATED_SMALL_CASE(DT, 1, 1, 4, 4)                                                                        \
    GP_GATED_SMALL_CASE(DT, 1, 1, 8, 4)                                                                        \
    GP_GATED_SMALL_CASE(DT, 2, 1, 4, 4)                                                                        \
    GP_GATED_SMALL_CASE(DT, 2, 1, 8, 4)                                                                        \
    GP_GATED_SMALL_CASE(DT, 4, 1, 8, 4)                                                                        \
    return hipErrorInvalidValue;                                                                               \
  }
