#include "linear_launch.cuh"

namespace maxsim {

template maxsim_status launch_tiles<int32_t>(const LinearPlan&, const LinearArgs&, const __half*, bool, int32_t*, const HostDevice&,
                                             cudaStream_t);

}  // namespace maxsim
