// Kernel instantiations of the linear layer with its epilogue for one input type.
#include "launch_linear.hpp"
#include "variants.hpp"

namespace gp {

GP_DEFINE_LINEAR(f16, DT_F16)

}  // namespace gp
