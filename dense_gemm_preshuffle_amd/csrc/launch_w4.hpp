// Launch tables of the 4-bit products.
#pragma once

#include "w4a16.hpp"

namespace gp {

// A variant of w4a16_kernel: x loads (0: one row, else rows / 4), column
// blocks, waves, 128-element K blocks per chunk.
struct W4Plan {
  int xl = 0, nb = 1, waves = 16, s = 1;
};
// sg: scales per 128-element block and column (1, 2, 4); _z: with zero points.
// hipErrorInvalidValue if the variant is not compiled.
hipError_t launch_w4_bf16(const W4Plan& p, int sg, const W4Args& a, hipStream_t s);
hipError_t launch_w4_bf16_z(const W4Plan& p, int sg, const W4Args& a, hipStream_t s);
hipError_t launch_w4_f16(const W4Plan& p, int sg, const W4Args& a, hipStream_t s);
hipError_t launch_w4_f16_z(const W4Plan& p, int sg, const W4Args& a, hipStream_t s);

}  // namespace gp

#define GP_W4_KERNEL(DT, XL, NB, W, S, SGV, ZV)                                                                \
  if (sg == SGV) {                                                                                             \
    constexpr uint32_t rows = XL == 0 ? 1 : 4 * XL;                                                            \
    const dim3 grid(((a.nblk + NB - 1) / NB) * ((a.M + rows - 1) / rows) * a.ksplit);                          \
    hipLaunchKernelGGL((w4a16_kernel<DT, XL, NB, W, S, SGV, ZV>), grid, dim3(W * 64), 0, s, a);                \
    return hipGetLastError();                                                                                  \
  }
#define GP_W4_CASE(DT, ZV, XL, NB, W, S)                                                                       \
  if (p.xl == XL && p.nb == NB && p.waves == W && p.s == S) {                                                  \
    GP_W4_KERNEL(DT, XL, NB, W, S, 1, ZV)                                                                      \
    GP_W4_KERNEL(DT, XL, NB, W, S, 2, ZV)                                                                      \
    GP_W4_KERNEL(DT, XL, NB, W, S, 4, ZV)                                                                      \
  }
#define GP_DEFINE_W4(NAME, DT, ZV)                                                                             \
  hipError_t launch_w4_##NAME(const W4Plan& p, int sg, const W4Args& a, hipStream_t s) {                       \
    GP_W4_CASE(DT, ZV, 0, 1, 16, 1)                                                                            \
    GP_W4_CASE(DT, ZV, 0, 2, 16, 1)                                                                            \
    GP_W4_CASE(DT, ZV, 0, 2, 8, 1)                                                                             \
    GP_W4_CASE(DT, ZV, 0, 2, 4, 2)                                                                             \
    GP_W4_CASE(DT, ZV, 1, 1, 16, 1)                                                                            \
    GP_W4_CASE(DT, ZV, 1, 2, 16, 1)                                                                            \
    GP_W4_CASE(DT, ZV, 1, 4, 4, 1)                                                                             \
    GP_W4_CASE(DT, ZV, 4, 1, 8, 1)                                                                             \
    GP_W4_CASE(DT, ZV, 4, 2, 8, 1)                                                                             \
    GP_W4_CASE(DT, ZV, 4, 4, 8, 1)                                                                             \
    GP_W4_CASE(DT, ZV, 8, 1, 8, 1)                                                                             \
    GP_W4_CASE(DT, ZV, 8, 2, 8, 1)                                                                             \
    GP_W4_CASE(DT, ZV, 8, 4, 8, 1)                                                                             \
    GP_W4_CASE(DT, ZV, 16, 1, 8, 1)                                                                            \
    GP_W4_CASE(DT, ZV, 16, 2, 4, 1)                                                                            \
    GP_W4_CASE(DT, ZV, 16, 4, 4, 1)                                                                            \
    return hipErrorInvalidValue;                                                                               \
  }
