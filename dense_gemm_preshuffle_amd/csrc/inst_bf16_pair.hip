// Both products of a backward pass in one kernel, for one input type.
#include "launch_rows.hpp"

namespace gp {

GP_DEFINE_PAIR(bf16, DT_BF16)

}  // namespace gp
