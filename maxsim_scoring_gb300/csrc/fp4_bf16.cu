#include "fp4_launch.cuh"

namespace maxsim {

template maxsim_status run_quantize_fp4<__nv_bfloat16>(const Fp4QuantizeArgs&, int, const HostDevice&, cudaStream_t);
template maxsim_status run_dequantize_fp4<__nv_bfloat16>(const Fp4DequantizeArgs&, int, const HostDevice&, cudaStream_t);

}  // namespace maxsim
