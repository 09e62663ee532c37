// Both products of a backward pass in one kernel, for one input type.
#include "launch_rows.hpp"

namespace gp {

GP_DEFINE_PAIR(f16, DT_F16)

}  // namespace gp
