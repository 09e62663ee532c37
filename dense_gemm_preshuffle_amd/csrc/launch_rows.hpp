// Launch tables of the tile kernel on a row-major B (BF16 and FP16).
#pragma once

#include "gemm_tile.hpp"

namespace gp {

// Each returns hipErrorInvalidValue if the variant is not compiled. _t: output
// stored transposed.
hipError_t launch_rows_bf16(int tm, int tn, const TileArgs& a, hipStream_t s);
hipError_t launch_rows_f16(int tm, int tn, const TileArgs& a, hipStream_t s);
hipError_t launch_rows_t_bf16(int tm, int tn, const TileArgs& a, hipStream_t s);
hipError_t launch_rows_t_f16(int tm, int tn, const TileArgs& a, hipStream_t s);

}  // namespace gp

#define GP_ROWS_CASE(DT, EPI, TM, TN, PIPE, KSV)                                                                   \
  if (tm == TM && tn == TN && (a.ksplit > 1) == KSV) {                                                         \
    hipLaunchKernelGGL((gemm_tile_kernel<DT, 16, TM, TN, 128, EPI, PIPE, false, 1, true, KSV>),                \
                       dim3(a.tiles_m * a.tiles_n * a.ksplit), dim3(64 * tile_waves(TM, TN)), 0, s, a);        \
    return hipGetLastError();                                                                                  \
  }
#define GP_DEFINE_ROWS(NAME, DT, EPI)                                                                          \
  hipError_t launch_rows##NAME(int tm, int tn, const TileArgs& a, hipStream_t s) {                             \
    GP_TILE_ROWS(GP_ROWS_CASE, DT, EPI)                                                                        \
    return hipErrorInvalidValue;                                                                               \
  }
