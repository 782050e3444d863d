// Row quantisation to INT8 and dropout (the token head's elementwise
// operators).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>

namespace maxsim {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// ---------------------------------------------------------------- row quantisation

// One block per row, two passes over it.
template <typename T>
__global__ void quantize_rows_kernel(const T* __restrict__ x, int64_t rows, int32_t cols, int64_t ld_x, int normalize,
                                     int8_t* __restrict__ q, int64_t ld_q, float* __restrict__ scale) {
    __shared__ uint32_t s_max[32];
    __shared__ float s_sum[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* xr = x + r * ld_x;
        // |x| as bits: ordered as the values, with infinities and NaN on top
        uint32_t m = 0;
        for (int32_t c = threadIdx.x; c < cols; c += blockDim.x)
            m = max(m, __float_as_uint(to_f32(xr[c])) & 0x7fffffffu);
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) s_max[warp] = m;
        __syncthreads();
        m = __reduce_max_sync(0xffffffffu, lane < warps ? s_max[lane] : 0u);
        const bool finite = m < 0x7f800000u;
        const float s = fmaxf(__fdiv_rn(__uint_as_float(m), 127.f), FLT_MIN);
        float sum = 0.f;
        for (int32_t c = threadIdx.x; c < cols; c += blockDim.x) {
            const float y = finite ? __fdiv_rn(to_f32(xr[c]), s) : 0.f;
            sum += y * y;
            q[r * ld_q + c] = static_cast<int8_t>(fminf(fmaxf(rintf(y), -127.f), 127.f));
        }
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            float total = 0.f;
            for (int w = 0; w < warps; ++w) total += s_sum[w];
            float out = s;
            if (normalize) out = total > 0.f ? __fdiv_rn(1.f, __fsqrt_rn(total)) : FLT_MIN;
            scale[r] = finite ? out : __uint_as_float(0x7fffffffu);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- dropout

// Philox4x32-10 (Salmon et al. 2011): ten rounds of two 32 x 32 -> 64 bit
// products, the key stepped by the Weyl constants.
__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = static_cast<uint64_t>(c.x) * 0xD2511F53u, b = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
        c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k0, static_cast<uint32_t>(b),
                       static_cast<uint32_t>(a >> 32) ^ c.w ^ k1, static_cast<uint32_t>(a));
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

struct DropoutArgs {
    const void* x;
    const void* residual;  // NULL = none
    void* y;
    int64_t rows, ld_x, ld_r, ld_y;
    int32_t cols;
    uint32_t drop;  // T: elements that draw less than this are dropped
    float scale;
    uint64_t seed, offset;
};

// One thread per counter value: eight elements of the row-major matrix.
template <typename T>
__global__ void dropout_kernel(const DropoutArgs a) {
    const int64_t n = a.rows * a.cols;
    const int64_t blocks = (n + 7) >> 3;
    const T* x = static_cast<const T*>(a.x);
    const T* res = static_cast<const T*>(a.residual);
    T* y = static_cast<T*>(a.y);
    for (int64_t b = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; b < blocks;
         b += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const uint4 u = philox4x32_10(
            make_uint4(static_cast<uint32_t>(b), static_cast<uint32_t>(static_cast<uint64_t>(b) >> 32),
                       static_cast<uint32_t>(a.offset), static_cast<uint32_t>(a.offset >> 32)),
            static_cast<uint32_t>(a.seed), static_cast<uint32_t>(a.seed >> 32));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        int64_t row = (b << 3) / a.cols;
        int32_t col = static_cast<int32_t>((b << 3) - row * a.cols);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if ((b << 3) + e >= n) break;
            const uint32_t bits = (e & 1) ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu;
            float v = bits >= a.drop ? to_f32(x[row * a.ld_x + col]) * a.scale : 0.f;
            if (res) v += to_f32(res[row * a.ld_r + col]);
            y[row * a.ld_y + col] = from_f32<T>(v);
            if (++col == a.cols) {
                col = 0;
                ++row;
            }
        }
    }
}

}  // namespace maxsim
