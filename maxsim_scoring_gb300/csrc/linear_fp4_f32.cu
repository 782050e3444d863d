#include "linear_fp4_launch.cuh"

namespace maxsim {

template maxsim_status run_linear_fp4<float>(const LinearFp4Plan&, const LinearFp4Args&, int, const HostDevice&, cudaStream_t);

}  // namespace maxsim
