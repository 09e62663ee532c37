// Kernel instantiations on a row-major B for one input type, transposed output.
#include "launch_rows.hpp"
#include "variants.hpp"

namespace gp {

GP_DEFINE_ROWS(_t_bf16, DT_BF16, EPI_ROWS_T)

}  // namespace gp
