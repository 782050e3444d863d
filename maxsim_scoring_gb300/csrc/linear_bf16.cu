#include "linear_launch.cuh"

namespace maxsim {

template maxsim_status run_linear<__nv_bfloat16>(const LinearPlan&, LinearArgs, bool, bool, uint8_t*, const HostDevice&, cudaStream_t);

}  // namespace maxsim
