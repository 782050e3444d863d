// out[m, n] = (sum_k x[m, k] w[n, k]) * x_scale[m] * w_scale[n] + bias[n] for
// rows of 4-bit floating-point values with block scales (fp4_kernels.cuh).
#pragma once

#include <cstdint>

#include "fp4_kernels.cuh"

namespace maxsim {

struct LinearFp4Args {
    const uint8_t* x;
    const uint8_t* w;
    const uint8_t* x_block;
    const uint8_t* w_block;
    int64_t ld_x, ld_w, ld_out;  // bytes, bytes, elements
    const float* x_scale;        // NULL: 1
    const float* w_scale;        // NULL: 1
    const float* bias;           // NULL: none
    void* out;
    int32_t M, N, K;             // K a multiple of 32
    int32_t words;               // scale words of a row
};

// A block of 16 x 16 outputs, one a thread, over pieces of 64 values.
template <typename T, int kBlock>
__global__ void __launch_bounds__(256) linear_fp4_simple_kernel(const LinearFp4Args a) {
    __shared__ float sx[16][65], sw[16][65];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t tiles_n = (a.N + 15) / 16, tiles = tiles_n * ((a.M + 15) / 16);
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t m0 = tile / tiles_n * 16, n0 = tile % tiles_n * 16;
        float sum = 0.f;
        for (int32_t k0 = 0; k0 < a.K; k0 += 64) {
            // thread t: four values of one of the 32 rows... each row 64 values, eight threads a row
            for (int i = threadIdx.x; i < 32 * 8; i += 256) {
                const int row = i >> 3, k = k0 + (i & 7) * 8;
                const bool is_x = row < 16;
                const int64_t r = is_x ? m0 + row : n0 + row - 16;
                float* to = is_x ? &sx[row][(i & 7) * 8] : &sw[row - 16][(i & 7) * 8];
                uint32_t h[4] = {0, 0, 0, 0};
                float b = 0.f;
                if (r < (is_x ? a.M : a.N) && k < a.K) {
                    from_e2m1x8(*reinterpret_cast<const uint32_t*>((is_x ? a.x + r * a.ld_x : a.w + r * a.ld_w) + k / 2), h);
                    b = block_scale_value<kBlock>((is_x ? a.x_block : a.w_block)[scale_word_at(r, k / (4 * kBlock), a.words) + (k / kBlock & 3)]);
                }
                for (int j = 0; j < 8; ++j)
                    to[j] = __half2float(__ushort_as_half(static_cast<unsigned short>(h[j >> 1] >> ((j & 1) * 16)))) * b;
            }
            __syncthreads();
            for (int k = 0; k < 64; ++k) sum = __fmaf_rn(sx[ty][k], sw[tx][k], sum);
            __syncthreads();
        }
        const int64_t m = m0 + ty, n = n0 + tx;
        if (m < a.M && n < a.N) {
            float y = sum * (a.x_scale ? a.x_scale[m] : 1.f) * (a.w_scale ? a.w_scale[n] : 1.f);
            if (a.bias) y += a.bias[n];
            static_cast<T*>(a.out)[m * a.ld_out + n] = from_f32<T>(y);
        }
    }
}

}  // namespace maxsim
