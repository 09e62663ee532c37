// Kernel instantiations of the linear layer with its epilogue for one input type.
#include "launch_linear.hpp"
#include "variants.hpp"

namespace gp {

GP_DEFINE_LINEAR(bf16, DT_BF16)

}  // namespace gp
