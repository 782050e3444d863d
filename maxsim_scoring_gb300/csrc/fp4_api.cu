// Host side of the 4-bit floating-point rows (include/maxsim.h): argument
// validation and the launches on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp4_launch.cuh"

namespace maxsim {

extern template maxsim_status run_quantize_fp4<__half>(const Fp4QuantizeArgs&, int, const HostDevice&, cudaStream_t);
extern template maxsim_status run_dequantize_fp4<__half>(const Fp4DequantizeArgs&, int, const HostDevice&, cudaStream_t);
extern template maxsim_status run_quantize_fp4<__nv_bfloat16>(const Fp4QuantizeArgs&, int, const HostDevice&, cudaStream_t);
extern template maxsim_status run_dequantize_fp4<__nv_bfloat16>(const Fp4DequantizeArgs&, int, const HostDevice&, cudaStream_t);
extern template maxsim_status run_quantize_fp4<float>(const Fp4QuantizeArgs&, int, const HostDevice&, cudaStream_t);
extern template maxsim_status run_dequantize_fp4<float>(const Fp4DequantizeArgs&, int, const HostDevice&, cudaStream_t);

namespace {

// Bytes of a row's codes, and its scale words.
inline int64_t code_bytes(int64_t cols) { return (cols + 31) / 32 * 16; }
inline int64_t scale_words(int64_t cols, int block) { return (cols + 4 * block - 1) / (4 * block); }

}  // namespace
}  // namespace maxsim

using namespace maxsim;

extern "C" {

maxsim_status maxsim_quantize_rows_fp4(const void* x, maxsim_dtype dtype, int64_t rows, int64_t cols, int64_t ld_x, int block,
                                       uint8_t* q, int64_t ld_q, uint8_t* block_scale, float* scale, void* stream) {
    if (!any_dtype(dtype) || rows < 0 || cols < 0 || (block != 16 && block != 32)) return MAXSIM_ERR_INVALID_ARG;
    if (!rows_fit(rows, cols, ld_x)) return MAXSIM_ERR_INVALID_ARG;
    if (rows > kI32Max - 127 || cols > kI32Max - 31) return MAXSIM_ERR_UNSUPPORTED;
    if (!rows_fit(rows, code_bytes(cols), ld_q) || (rows > 1 && ld_q % 16 != 0)) return MAXSIM_ERR_INVALID_ARG;
    if (rows == 0) return MAXSIM_OK;
    if (block == 16 && (!scale || !ptr_aligned(scale, 4))) return MAXSIM_ERR_INVALID_ARG;
    if (cols > 0 && (!x || !q || !block_scale || !ptr_aligned(x, elem_bytes(dtype)) || !ptr_aligned(q, 16) || !ptr_aligned(block_scale, 16)))
        return MAXSIM_ERR_INVALID_ARG;
    HostDevice dev;
    const maxsim_status rc = host_device(&dev);
    if (rc != MAXSIM_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Fp4QuantizeArgs a{x, q, block_scale, scale, rows, ld_x, ld_q, static_cast<int32_t>(cols),
                            static_cast<int32_t>(code_bytes(cols) / 8), static_cast<int32_t>(scale_words(cols, block))};
    if (dtype == MAXSIM_F16) return run_quantize_fp4<__half>(a, block, dev, st);
    if (dtype == MAXSIM_BF16) return run_quantize_fp4<__nv_bfloat16>(a, block, dev, st);
    return run_quantize_fp4<float>(a, block, dev, st);
}

maxsim_status maxsim_dequantize_rows_fp4(const uint8_t* q, int64_t ld_q, const uint8_t* block_scale, const float* scale,
                                         int64_t rows, int64_t cols, int block, maxsim_dtype out_dtype, void* y, int64_t ld_y,
                                         void* stream) {
    if (!any_dtype(out_dtype) || rows < 0 || cols < 0 || (block != 16 && block != 32)) return MAXSIM_ERR_INVALID_ARG;
    if (!rows_fit(rows, cols, ld_y)) return MAXSIM_ERR_INVALID_ARG;
    if (rows > kI32Max - 127 || cols > kI32Max - 31) return MAXSIM_ERR_UNSUPPORTED;
    if (!rows_fit(rows, code_bytes(cols), ld_q) || (rows > 1 && ld_q % 16 != 0)) return MAXSIM_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return MAXSIM_OK;
    if (!q || !block_scale || !y || !ptr_aligned(q, 16) || !ptr_aligned(block_scale, 16) || !ptr_aligned(scale, 4) ||
        !ptr_aligned(y, elem_bytes(out_dtype)))
        return MAXSIM_ERR_INVALID_ARG;
    HostDevice dev;
    const maxsim_status rc = host_device(&dev);
    if (rc != MAXSIM_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Fp4DequantizeArgs a{q, block_scale, scale, y, rows, ld_q, ld_y, static_cast<int32_t>(cols),
                              static_cast<int32_t>(scale_words(cols, block))};
    if (out_dtype == MAXSIM_F16) return run_dequantize_fp4<__half>(a, block, dev, st);
    if (out_dtype == MAXSIM_BF16) return run_dequantize_fp4<__nv_bfloat16>(a, block, dev, st);
    return run_dequantize_fp4<float>(a, block, dev, st);
}

}  // extern "C"
