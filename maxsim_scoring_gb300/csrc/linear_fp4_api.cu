// Host side of the 4-bit linear (include/maxsim.h): argument validation and
// the launches on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "maxsim.h"
#include "host_util.h"
#include "linear_fp4.cuh"

namespace maxsim {
namespace {

constexpr int64_t kMaxRows = kI32Max - 1023;  // a tile past the last row still has 32-bit coordinates

template <typename T>
maxsim_status run_linear_fp4(const LinearFp4Args& a, int block, const HostDevice& dev, cudaStream_t st) {
    const unsigned grid = grid_of((int64_t(a.M) + 15) / 16 * ((int64_t(a.N) + 15) / 16), 1, int64_t(dev.num_sms) * 64);
    if (block == 16) linear_fp4_simple_kernel<T, 16><<<grid, 256, 0, st>>>(a);
    else linear_fp4_simple_kernel<T, 32><<<grid, 256, 0, st>>>(a);
    return launched();
}

}  // namespace
}  // namespace maxsim

using namespace maxsim;

extern "C" {

maxsim_status maxsim_linear_fp4(const uint8_t* x, int64_t ld_x, const uint8_t* x_block_scale, const float* x_scale,
                                const uint8_t* w, int64_t ld_w, const uint8_t* w_block_scale, const float* w_scale,
                                const float* bias, int64_t M, int64_t N, int64_t K, int block, maxsim_dtype out_dtype,
                                void* out, int64_t ld_out, void* stream) {
    if (!any_dtype(out_dtype) || M < 0 || N < 0 || K < 0 || (block != 16 && block != 32)) return MAXSIM_ERR_INVALID_ARG;
    if (K % 32 != 0 || !rows_fit(M, K / 2, ld_x) || !rows_fit(N, K / 2, ld_w) || !rows_fit(M, N, ld_out)) return MAXSIM_ERR_INVALID_ARG;
    if (M > kMaxRows || N > kMaxRows || K > kI32Max - 1023) return MAXSIM_ERR_UNSUPPORTED;
    if ((M > 1 && ld_x % 16 != 0) || (N > 1 && ld_w % 16 != 0)) return MAXSIM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return MAXSIM_OK;
    if (!out || !ptr_aligned(out, elem_bytes(out_dtype)) || !ptr_aligned(x_scale, 4) || !ptr_aligned(w_scale, 4) || !ptr_aligned(bias, 4))
        return MAXSIM_ERR_INVALID_ARG;
    if (K > 0 && (!x || !w || !x_block_scale || !w_block_scale)) return MAXSIM_ERR_INVALID_ARG;
    if (!ptr_aligned(x, 16) || !ptr_aligned(w, 16) || !ptr_aligned(x_block_scale, 16) || !ptr_aligned(w_block_scale, 16))
        return MAXSIM_ERR_INVALID_ARG;
    HostDevice dev;
    const maxsim_status rc = host_device(&dev);
    if (rc != MAXSIM_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const LinearFp4Args a{x, w, x_block_scale, w_block_scale, ld_x, ld_w, ld_out, x_scale, w_scale, bias, out,
                          static_cast<int32_t>(M), static_cast<int32_t>(N), static_cast<int32_t>(K),
                          static_cast<int32_t>((K + 4 * block - 1) / (4 * block))};
    if (out_dtype == MAXSIM_F16) return run_linear_fp4<__half>(a, block, dev, st);
    if (out_dtype == MAXSIM_BF16) return run_linear_fp4<__nv_bfloat16>(a, block, dev, st);
    return run_linear_fp4<float>(a, block, dev, st);
}

}  // extern "C"
