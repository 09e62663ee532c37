// Kernel instantiations of the 4-bit products for one input type, without zero points.
#include "launch_w4.hpp"

namespace gp {

GP_DEFINE_W4(bf16, DT_BF16, false)

}  // namespace gp
