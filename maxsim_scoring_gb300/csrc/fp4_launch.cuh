// Launches of the 4-bit rows' kernels, per element type (fp4_f16.cu, fp4_bf16.cu,
// fp4_f32.cu, compiled side by side).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "maxsim.h"
#include "host_util.h"
#include "fp4_kernels.cuh"

namespace maxsim {

template <typename T, int kBlock, bool kWide, int kGroup, int kChunks>
maxsim_status launch_group(const Fp4QuantizeArgs& a, const HostDevice& dev, cudaStream_t st) {
    constexpr int kThreads = fp4_threads(kGroup), kRows = kThreads / kGroup, kTile = 128 / kRows;  // kTile: blocks of 128 rows
    const int64_t tiles = (a.rows + 127) / 128, most = (int64_t(dev.num_sms) * (2048 / kThreads) + kTile - 1) / kTile;
    fp4_quantize_kernel<T, kBlock, kWide, kGroup, kChunks><<<grid_of(tiles, 1, most) * kTile, kThreads, 0, st>>>(a);
    return launched();
}

// The smallest group of threads that holds a row's chunks of 16 elements.
template <typename T, int kBlock, bool kWide>
maxsim_status launch_quantize(const Fp4QuantizeArgs& a, const HostDevice& dev, cudaStream_t st) {
    if (a.chunks <= 2) return launch_group<T, kBlock, kWide, 2, 1>(a, dev, st);
    if (a.chunks <= 4) return launch_group<T, kBlock, kWide, 4, 1>(a, dev, st);
    if (a.chunks <= 8) return launch_group<T, kBlock, kWide, 8, 1>(a, dev, st);
    if (a.chunks <= 16) return launch_group<T, kBlock, kWide, 16, 1>(a, dev, st);
    if (a.chunks <= 32) return launch_group<T, kBlock, kWide, 32, 1>(a, dev, st);
    if (a.chunks <= 64) return launch_group<T, kBlock, kWide, 32, 2>(a, dev, st);
    if (a.chunks <= 96) return launch_group<T, kBlock, kWide, 32, 3>(a, dev, st);
    if (a.chunks <= 128) return launch_group<T, kBlock, kWide, 64, 2>(a, dev, st);
    if (a.chunks <= 192) return launch_group<T, kBlock, kWide, 64, 3>(a, dev, st);
    if (a.chunks <= 256) return launch_group<T, kBlock, kWide, 128, 2>(a, dev, st);
    if (a.chunks <= 512) return launch_group<T, kBlock, kWide, 256, 2>(a, dev, st);
    if (a.chunks <= 1024) return launch_group<T, kBlock, kWide, 512, 2>(a, dev, st);
    fp4_quantize_long_kernel<T, kBlock, kWide>
        <<<grid_of((a.rows + 127) / 128 * 128, 1, int64_t(dev.num_sms) * 4), 512, 0, st>>>(a);
    return launched();
}

template <typename T>
maxsim_status run_quantize_fp4(const Fp4QuantizeArgs& a, int block, const HostDevice& dev, cudaStream_t st) {
    const bool wide = ptr_aligned(a.x, 32) && (a.rows == 1 || a.ld_x * static_cast<int64_t>(sizeof(T)) % 32 == 0);
    if (block == 16) return wide ? launch_quantize<T, 16, true>(a, dev, st) : launch_quantize<T, 16, false>(a, dev, st);
    return wide ? launch_quantize<T, 32, true>(a, dev, st) : launch_quantize<T, 32, false>(a, dev, st);
}

template <typename T, int kBlock, bool kWide, int kGroup, bool kRowsAhead>
void launch_dequantize_group(const Fp4DequantizeArgs& a, const HostDevice& dev, cudaStream_t st) {
    constexpr int kRows = 256 / kGroup;
    // few rows: every block one round of them
    const int64_t most = int64_t(dev.num_sms) * 16, blocks = (a.rows + kRows - 1) / kRows;
    fp4_dequantize_kernel<T, kBlock, kWide, kGroup, kRowsAhead><<<static_cast<unsigned>(std::min(blocks, most)), 256, 0, st>>>(a);
}

template <typename T, int kBlock, bool kWide>
maxsim_status launch_dequantize(const Fp4DequantizeArgs& a, const HostDevice& dev, cudaStream_t st) {
    if (a.cols <= 32) launch_dequantize_group<T, kBlock, kWide, 2, true>(a, dev, st);
    else if (a.cols <= 64) launch_dequantize_group<T, kBlock, kWide, 4, true>(a, dev, st);
    else if (a.cols <= 128) launch_dequantize_group<T, kBlock, kWide, 8, true>(a, dev, st);
    else if (a.cols <= 256) launch_dequantize_group<T, kBlock, kWide, 16, true>(a, dev, st);
    else if (a.cols <= 512) launch_dequantize_group<T, kBlock, kWide, 32, true>(a, dev, st);
    else if (a.cols <= 1024) launch_dequantize_group<T, kBlock, kWide, 64, true>(a, dev, st);
    else if (a.cols <= 2048) launch_dequantize_group<T, kBlock, kWide, 128, true>(a, dev, st);
    else if (a.cols <= 4096) launch_dequantize_group<T, kBlock, kWide, 256, true>(a, dev, st);
    else launch_dequantize_group<T, kBlock, kWide, 256, false>(a, dev, st);
    return launched();
}

template <typename T>
maxsim_status run_dequantize_fp4(const Fp4DequantizeArgs& a, int block, const HostDevice& dev, cudaStream_t st) {
    const bool wide = ptr_aligned(a.y, 32) && (a.rows == 1 || a.ld_y * static_cast<int64_t>(sizeof(T)) % 32 == 0);
    if (block == 16) return wide ? launch_dequantize<T, 16, true>(a, dev, st) : launch_dequantize<T, 16, false>(a, dev, st);
    return wide ? launch_dequantize<T, 32, true>(a, dev, st) : launch_dequantize<T, 32, false>(a, dev, st);
}

}  // namespace maxsim
