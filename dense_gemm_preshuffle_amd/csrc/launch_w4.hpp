// Launch tables of the 4-bit products.
#pragma once

#include "w4a16.hpp"

namespace gp {

// A variant: row blocks, column blocks, waves, 128-element K blocks per chunk.
struct W4Plan {
  int mb = 1, nb = 1, waves = 8;
  bool one = false;   // a single row
};
// sg: scales per 128-element block and column (1, 2, 4). hipErrorInvalidValue
// if the variant is not compiled.
hipError_t launch_w4_bf16(const W4Plan& p, int sg, const W4Args& a, hipStream_t s);
hipError_t launch_w4_f16(const W4Plan& p, int sg, const W4Args& a, hipStream_t s);

}  // namespace gp

#define GP_W4_KERNEL(DT, MB, NB, W, S, SGV, ZV, ONE)                                                              \
  {                                                                                                            \
    const dim3 grid(((a.nblk + NB - 1) / NB) * ((a.M + 16 * MB - 1) / (16 * MB)));                              \
    hipLaunchKernelGGL((w4a16_kernel<DT, MB, NB, W, S, SGV, ZV, ONE>), grid, dim3(W * 64), 0, s, a);            \
    return hipGetLastError();                                                                                  \
  }
#define GP_W4_CASE(DT, MB, NB, W, S, ONE)                                                                      \
  if (p.mb == MB && p.nb == NB && p.waves == W && p.one == ONE) {                                              \
    if (sg == 1 && !a.z) GP_W4_KERNEL(DT, MB, NB, W, S, 1, false, ONE)                                         \
    if (sg == 2 && !a.z) GP_W4_KERNEL(DT, MB, NB, W, S, 2, false, ONE)                                         \
    if (sg == 4 && !a.z) GP_W4_KERNEL(DT, MB, NB, W, S, 4, false, ONE)                                         \
    if (sg == 1) GP_W4_KERNEL(DT, MB, NB, W, S, 1, true, ONE)                                                  \
    if (sg == 2) GP_W4_KERNEL(DT, MB, NB, W, S, 2, true, ONE)                                                  \
    if (sg == 4) GP_W4_KERNEL(DT, MB, NB, W, S, 4, true, ONE)                                                  \
  }
// (rows / 16, columns / 16, waves, K blocks per chunk, single row)
#define GP_DEFINE_W4(NAME, DT)                                                                                 \
  hipError_t launch_w4_##NAME(const W4Plan& p, int sg, const W4Args& a, hipStream_t s) {                       \
    GP_W4_CASE(DT, 1, 1, 8, 2, true)                                                                           \
    GP_W4_CASE(DT, 1, 2, 8, 2, true)                                                                           \
    GP_W4_CASE(DT, 1, 1, 8, 2, false)                                                                          \
    GP_W4_CASE(DT, 1, 2, 8, 2, false)                                                                          \
    GP_W4_CASE(DT, 2, 2, 8, 1, false)                                                                          \
    return hipErrorInvalidValue;                                                                               \
  }
