// Host side of the 4-bit linear (include/maxsim.h): argument validation and
// the launches on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "linear_fp4_launch.cuh"

namespace maxsim {

extern template maxsim_status run_linear_fp4<__half>(const LinearFp4Plan&, const LinearFp4Args&, int, const HostDevice&, cudaStream_t);
extern template maxsim_status run_linear_fp4<__nv_bfloat16>(const LinearFp4Plan&, const LinearFp4Args&, int, const HostDevice&, cudaStream_t);
extern template maxsim_status run_linear_fp4<float>(const LinearFp4Plan&, const LinearFp4Args&, int, const HostDevice&, cudaStream_t);

namespace {

constexpr int64_t kMaxRows = kI32Max - 1023;  // a tile past the last row still has 32-bit coordinates
constexpr int64_t kMaxK = int64_t(1) << 28;   // a tile's sums (a million stages) take well below the limit of a wait
constexpr int64_t kMaxStride = int64_t(1) << 40;  // of a TMA descriptor

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
    if (M > kMaxRows || N > kMaxRows || K > kMaxK) return MAXSIM_ERR_UNSUPPORTED;
    if ((M > 1 && ld_x >= kMaxStride) || (N > 1 && ld_w >= kMaxStride)) return MAXSIM_ERR_UNSUPPORTED;
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
    const LinearFp4Plan p = plan_linear_fp4(M, N, K);
    if (p.tiles > kI32Max) return MAXSIM_ERR_UNSUPPORTED;
    if (out_dtype == MAXSIM_F16) return run_linear_fp4<__half>(p, a, block, dev, st);
    if (out_dtype == MAXSIM_BF16) return run_linear_fp4<__nv_bfloat16>(p, a, block, dev, st);
    return run_linear_fp4<float>(p, a, block, dev, st);
}

}  // extern "C"
