#include "fp4_launch.cuh"

namespace maxsim {

template maxsim_status run_quantize_fp4<__half>(const Fp4QuantizeArgs&, int, const HostDevice&, cudaStream_t);
template maxsim_status run_dequantize_fp4<__half>(const Fp4DequantizeArgs&, int, const HostDevice&, cudaStream_t);

}  // namespace maxsim
