// Host side of the token head's entry points (include/maxsim.h): argument
// validation and the launches on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "maxsim.h"
#include "host_util.h"
#include "head_kernels.cuh"
#include "linear_int8.cuh"

namespace maxsim {
namespace {

constexpr int64_t kI32Max = 2147483647;
constexpr int64_t kLinearMaxK = 131071;  // 131071 * 128 * 128 < 2^31

inline int elem_bytes(maxsim_dtype t) { return t == MAXSIM_F32 ? 4 : 2; }
inline bool any_dtype(maxsim_dtype t) { return t == MAXSIM_F16 || t == MAXSIM_BF16 || t == MAXSIM_F32; }

inline unsigned grid_of(int64_t items, int64_t per_block, int64_t most) {
    return static_cast<unsigned>(std::max<int64_t>(1, std::min((items + per_block - 1) / per_block, most)));
}

inline maxsim_status launched() { return cudaGetLastError() == cudaSuccess ? MAXSIM_OK : MAXSIM_ERR_CUDA; }

// A [rows, cols] operand with rows ld elements apart whose bytes can be addressed with 64 bits.
inline bool rows_fit(int64_t rows, int64_t cols, int64_t ld) {
    return ld >= cols && (rows <= 1 || ld <= (int64_t(1) << 60) / std::max<int64_t>(rows, 1));
}

template <typename T>
maxsim_status launch_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld_x, int normalize, int8_t* q,
                              int64_t ld_q, float* scale, const HostDevice& dev, cudaStream_t st) {
    quantize_rows_kernel<T><<<grid_of(rows, 1, int64_t(dev.num_sms) * 8), 256, 0, st>>>(
        static_cast<const T*>(x), rows, static_cast<int32_t>(cols), ld_x, normalize, q, ld_q, scale);
    return launched();
}

maxsim_status run_dropout(const DropoutArgs& a, maxsim_dtype dtype, cudaStream_t st) {
    HostDevice dev;
    const maxsim_status rc = host_device(&dev);
    if (rc != MAXSIM_OK) return rc;
    const int64_t blocks = (a.rows * a.cols + 7) / 8;
    const unsigned grid = grid_of(blocks, 256, int64_t(dev.num_sms) * 8);
    if (dtype == MAXSIM_F16) dropout_kernel<__half><<<grid, 256, 0, st>>>(a);
    else if (dtype == MAXSIM_BF16) dropout_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
    else dropout_kernel<float><<<grid, 256, 0, st>>>(a);
    return launched();
}

// Fills drop and scale from p; false where p is no probability.
bool dropout_rate(double p, DropoutArgs* a) {
    if (!(p >= 0.0 && p <= 1.0)) return false;
    const uint32_t t = static_cast<uint32_t>(std::nearbyint(p * 65536.0));
    a->drop = t;
    a->scale = t < 65536u ? static_cast<float>(65536.0 / (65536.0 - t)) : 0.f;
    return true;
}

}  // namespace

size_t linear_int8_ws_bytes(int64_t M, int64_t N, int64_t K, int64_t ld_x, int64_t ld_w) {
    if (M < 0 || N < 0 || K < 0 || ld_x < 0 || ld_w < 0 || M > kI32Max || N > kI32Max || K > kLinearMaxK)
        return static_cast<size_t>(-1);
    return 0;
}

}  // namespace maxsim

using namespace maxsim;

extern "C" {

maxsim_status maxsim_quantize_rows(const void* x, maxsim_dtype dtype, int64_t rows, int64_t cols, int64_t ld_x,
                                   int normalize, int8_t* q, int64_t ld_q, float* scale, void* stream) {
    if (!any_dtype(dtype) || rows < 0 || cols < 0) return MAXSIM_ERR_INVALID_ARG;
    if (!rows_fit(rows, cols, ld_x) || !rows_fit(rows, cols, ld_q)) return MAXSIM_ERR_INVALID_ARG;
    if (rows > kI32Max || cols > kI32Max) return MAXSIM_ERR_UNSUPPORTED;
    if (rows == 0) return MAXSIM_OK;
    if (!scale || !ptr_aligned(scale, 4)) return MAXSIM_ERR_INVALID_ARG;
    if (cols > 0 && (!x || !q || !ptr_aligned(x, elem_bytes(dtype)))) return MAXSIM_ERR_INVALID_ARG;
    HostDevice dev;
    const maxsim_status rc = host_device(&dev);
    if (rc != MAXSIM_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == MAXSIM_F16) return launch_quantize<__half>(x, rows, cols, ld_x, normalize, q, ld_q, scale, dev, st);
    if (dtype == MAXSIM_BF16)
        return launch_quantize<__nv_bfloat16>(x, rows, cols, ld_x, normalize, q, ld_q, scale, dev, st);
    return launch_quantize<float>(x, rows, cols, ld_x, normalize, q, ld_q, scale, dev, st);
}

maxsim_status maxsim_linear_int8(const int8_t* x, int64_t ld_x, const float* x_scale, const int8_t* w, int64_t ld_w,
                                 const float* w_scale, const float* bias, int64_t M, int64_t N, int64_t K,
                                 maxsim_dtype out_dtype, void* out, int64_t ld_out, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    if (!any_dtype(out_dtype) || M < 0 || N < 0 || K < 0) return MAXSIM_ERR_INVALID_ARG;
    if (!rows_fit(M, K, ld_x) || !rows_fit(N, K, ld_w) || !rows_fit(M, N, ld_out)) return MAXSIM_ERR_INVALID_ARG;
    if (M > kI32Max || N > kI32Max || K > kLinearMaxK) return MAXSIM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return MAXSIM_OK;
    if (!out || !ptr_aligned(out, elem_bytes(out_dtype))) return MAXSIM_ERR_INVALID_ARG;
    if (!x_scale || !w_scale || !ptr_aligned(x_scale, 4) || !ptr_aligned(w_scale, 4) || !ptr_aligned(bias, 4))
        return MAXSIM_ERR_INVALID_ARG;
    if (K > 0 && (!x || !w)) return MAXSIM_ERR_INVALID_ARG;
    HostDevice dev;
    const maxsim_status rc = host_device(&dev);
    if (rc != MAXSIM_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    LinearArgs a{x, w, ld_x, ld_w, ld_out, x_scale, w_scale, bias, out,
                 static_cast<int32_t>(M), static_cast<int32_t>(N), static_cast<int32_t>(K)};
    const unsigned grid = grid_of(((M + 15) / 16) * ((N + 15) / 16), 1, int64_t(dev.num_sms) * 8);
    if (out_dtype == MAXSIM_F16) linear_simple_kernel<__half><<<grid, 256, 0, st>>>(a);
    else if (out_dtype == MAXSIM_BF16) linear_simple_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
    else linear_simple_kernel<float><<<grid, 256, 0, st>>>(a);
    return launched();
}

maxsim_status maxsim_dropout_fwd(const void* x, maxsim_dtype dtype, int64_t rows, int64_t cols, int64_t ld_x,
                                 const void* residual, int64_t ld_residual, double p, uint64_t seed, uint64_t offset,
                                 void* y, int64_t ld_y, void* stream) {
    DropoutArgs a{};
    if (!any_dtype(dtype) || rows < 0 || cols < 0 || !dropout_rate(p, &a)) return MAXSIM_ERR_INVALID_ARG;
    if (!rows_fit(rows, cols, ld_x) || !rows_fit(rows, cols, ld_y)) return MAXSIM_ERR_INVALID_ARG;
    if (residual && !rows_fit(rows, cols, ld_residual)) return MAXSIM_ERR_INVALID_ARG;
    if (rows > kI32Max || cols > kI32Max) return MAXSIM_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return MAXSIM_OK;
    const int e = elem_bytes(dtype);
    if (!x || !y || !ptr_aligned(x, e) || !ptr_aligned(y, e) || !ptr_aligned(residual, e))
        return MAXSIM_ERR_INVALID_ARG;
    a.x = x;
    a.residual = residual;
    a.y = y;
    a.rows = rows;
    a.cols = static_cast<int32_t>(cols);
    a.ld_x = ld_x;
    a.ld_r = ld_residual;
    a.ld_y = ld_y;
    a.seed = seed;
    a.offset = offset;
    return run_dropout(a, dtype, static_cast<cudaStream_t>(stream));
}

maxsim_status maxsim_dropout_bwd(const void* grad, maxsim_dtype dtype, int64_t rows, int64_t cols, int64_t ld_grad,
                                 double p, uint64_t seed, uint64_t offset, void* dx, int64_t ld_dx, void* stream) {
    // the mask is the forward's, drawn again: the same map without a residual
    return maxsim_dropout_fwd(grad, dtype, rows, cols, ld_grad, nullptr, 0, p, seed, offset, dx, ld_dx, stream);
}

}  // extern "C"
