// out[m, n] = (sum_k x[m, k] w[n, k]) * x_scale[m] * w_scale[n] + bias[n] for
// 8-bit integers x [M, K] and w [N, K].
#pragma once

#include <cstdint>

#include "head_kernels.cuh"

namespace maxsim {

struct LinearArgs {
    const int8_t* x;
    const int8_t* w;
    int64_t ld_x, ld_w, ld_out;
    const float* x_scale;
    const float* w_scale;
    const float* bias;  // NULL = none
    void* out;
    int32_t M, N, K;
};

// 16 x 16 outputs per block, operands through shared memory.
template <typename T>
__global__ void linear_simple_kernel(const LinearArgs a) {
    __shared__ int8_t sx[16][68], sw[16][68];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t tiles_n = (static_cast<int64_t>(a.N) + 15) / 16;
    const int64_t tiles = tiles_n * ((static_cast<int64_t>(a.M) + 15) / 16);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t m0 = t / tiles_n * 16, n0 = t % tiles_n * 16;
        int32_t acc = 0;
        for (int32_t k0 = 0; k0 < a.K; k0 += 64) {
            for (int i = threadIdx.x; i < 16 * 64; i += blockDim.x) {
                const int r = i >> 6, k = i & 63;
                const bool in = k0 + k < a.K;
                sx[r][k] = in && m0 + r < a.M ? a.x[(m0 + r) * a.ld_x + k0 + k] : static_cast<int8_t>(0);
                sw[r][k] = in && n0 + r < a.N ? a.w[(n0 + r) * a.ld_w + k0 + k] : static_cast<int8_t>(0);
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 64; k += 4)
                acc = __dp4a(*reinterpret_cast<const int*>(&sx[ty][k]), *reinterpret_cast<const int*>(&sw[tx][k]), acc);
            __syncthreads();
        }
        const int64_t m = m0 + ty, n = n0 + tx;
        if (m < a.M && n < a.N) {
            float v = static_cast<float>(acc) * a.x_scale[m] * a.w_scale[n];
            if (a.bias) v += a.bias[n];
            static_cast<T*>(a.out)[m * a.ld_out + n] = from_f32<T>(v);
        }
    }
}

}  // namespace maxsim
