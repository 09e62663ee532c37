// Kernel instantiations of the 4-bit products for one input type, without zero points.
#include "launch_w4.hpp"

namespace gp {

GP_DEFINE_W4(f16, DT_F16, false)

}  // namespace gp
