// Kernel instantiations on a row-major B for one input type.
#include "launch_rows.hpp"
#include "variants.hpp"

namespace gp {

GP_DEFINE_ROWS(_bf16, DT_BF16, EPI_ROWS)

}  // namespace gp
