// Kernel instantiations of the 4-bit products for one input type, with zero points.
#include "launch_w4.hpp"

namespace gp {

GP_DEFINE_W4(bf16_z, DT_BF16, true)

}  // namespace gp
