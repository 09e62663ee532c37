// Kernel instantiations on a row-major B for one input type, transposed output.
#include "launch_rows.hpp"
#include "variants.hpp"

namespace gp {

GP_DEFINE_ROWS(_t_f16, DT_F16, EPI_ROWS_T)

}  // namespace gp
