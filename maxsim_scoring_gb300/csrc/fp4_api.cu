// Host side of the 4-bit floating-point rows (include/maxsim.h): argument
// validation and the launches on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "maxsim.h"
#include "host_util.h"
#include "fp4_kernels.cuh"

namespace maxsim {
namespace {

template <typename T, int kBlock, bool kWide, int kGroup, int kChunks>
maxsim_status launch_group(const Fp4QuantizeArgs& a, const HostDevice& dev, cudaStream_t st) {
    constexpr int kThreads = fp4_threads(kGroup);
    const int64_t padded = (a.rows + 127) / 128 * 128;
    fp4_quantize_kernel<T, kBlock, kWide, kGroup, kChunks>
        <<<grid_of(padded, kThreads / kGroup, int64_t(dev.num_sms) * (2048 / kThreads)), kThreads, 0, st>>>(a);
    return launched();
}

// The smallest group of threads that holds a row's chunks of 16 elements.
template <typename T, int kBlock, bool kWide>
maxsim_status launch_quantize(const Fp4QuantizeArgs& a, const HostDevice& dev, cudaStream_t st) {
    if (a.chunks <= 2) return launch_group<T, kBlock, kWide, 2, 1>(a, dev, st);
    if (a.chunks <= 8) return launch_group<T, kBlock, kWide, 8, 1>(a, dev, st);
    if (a.chunks <= 32) return launch_group<T, kBlock, kWide, 32, 1>(a, dev, st);
    if (a.chunks <= 64) return launch_group<T, kBlock, kWide, 32, 2>(a, dev, st);
    if (a.chunks <= 128) return launch_group<T, kBlock, kWide, 64, 2>(a, dev, st);
    if (a.chunks <= 256) return launch_group<T, kBlock, kWide, 128, 2>(a, dev, st);
    if (a.chunks <= 512) return launch_group<T, kBlock, kWide, 256, 2>(a, dev, st);
    if (a.chunks <= 1024) return launch_group<T, kBlock, kWide, 512, 2>(a, dev, st);
    fp4_quantize_long_kernel<T, kBlock, kWide>
        <<<grid_of((a.rows + 127) / 128 * 128, 1, int64_t(dev.num_sms) * 4), 512, 0, st>>>(a);
    return launched();
}

template <typename T>
maxsim_status run_quantize(const Fp4QuantizeArgs& a, int block, const HostDevice& dev, cudaStream_t st) {
    const bool wide = ptr_aligned(a.x, 32) && (a.rows == 1 || a.ld_x * static_cast<int64_t>(sizeof(T)) % 32 == 0);
    if (block == 16) return wide ? launch_quantize<T, 16, true>(a, dev, st) : launch_quantize<T, 16, false>(a, dev, st);
    return wide ? launch_quantize<T, 32, true>(a, dev, st) : launch_quantize<T, 32, false>(a, dev, st);
}

template <typename T, int kBlock, bool kWide>
maxsim_status launch_dequantize(const Fp4DequantizeArgs& a, const HostDevice& dev, cudaStream_t st) {
    const int64_t most = int64_t(dev.num_sms) * 8;
    if (a.cols <= 128) fp4_dequantize_kernel<T, kBlock, kWide, 8><<<grid_of(a.rows, 32, most), 256, 0, st>>>(a);
    else if (a.cols <= 1024) fp4_dequantize_kernel<T, kBlock, kWide, 32><<<grid_of(a.rows, 8, most), 256, 0, st>>>(a);
    else fp4_dequantize_kernel<T, kBlock, kWide, 256><<<grid_of(a.rows, 1, most), 256, 0, st>>>(a);
    return launched();
}

template <typename T>
maxsim_status run_dequantize(const Fp4DequantizeArgs& a, int block, const HostDevice& dev, cudaStream_t st) {
    const bool wide = ptr_aligned(a.y, 32) && (a.rows == 1 || a.ld_y * static_cast<int64_t>(sizeof(T)) % 32 == 0);
    if (block == 16) return wide ? launch_dequantize<T, 16, true>(a, dev, st) : launch_dequantize<T, 16, false>(a, dev, st);
    return wide ? launch_dequantize<T, 32, true>(a, dev, st) : launch_dequantize<T, 32, false>(a, dev, st);
}

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
    if (dtype == MAXSIM_F16) return run_quantize<__half>(a, block, dev, st);
    if (dtype == MAXSIM_BF16) return run_quantize<__nv_bfloat16>(a, block, dev, st);
    return run_quantize<float>(a, block, dev, st);
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
    if (out_dtype == MAXSIM_F16) return run_dequantize<__half>(a, block, dev, st);
    if (out_dtype == MAXSIM_BF16) return run_dequantize<__nv_bfloat16>(a, block, dev, st);
    return run_dequantize<float>(a, block, dev, st);
}

}  // extern "C"
