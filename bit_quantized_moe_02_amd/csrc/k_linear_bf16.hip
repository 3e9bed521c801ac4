// moe_linear for rows of type MOE_DT_BF16 (the kernel: linear_common.hpp).
#include "linear_common.hpp"

namespace qmoe {

template hipError_t launch_linear_type<MOE_DT_BF16>(const LinearArgs&, int, int, hipStream_t);

}  // namespace qmoe
