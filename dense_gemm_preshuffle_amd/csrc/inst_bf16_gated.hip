// Kernel instantiations with the gated epilogue for one input type.
#include "launch_gated.hpp"
#include "variants.hpp"

namespace gp {

GP_DEFINE_GATED(bf16, DT_BF16)

}  // namespace gp
