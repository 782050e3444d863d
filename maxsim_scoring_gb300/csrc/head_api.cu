// Host side of the row quantisation and dropout (include/maxsim.h): argument
// validation and the launches on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "maxsim.h"
#include "host_util.h"
#include "head_kernels.cuh"

namespace maxsim {
namespace {

template <typename T, RowMode kMode, bool kNorm, int kGroup, int kChunks>
maxsim_status launch_quantize_group(const QuantizeArgs& a, const HostDevice& dev, cudaStream_t st) {
    constexpr int kThreads = quantize_threads(kGroup);
    const unsigned grid = grid_of(a.rows, kThreads / kGroup, int64_t(dev.num_sms) * (2048 / kThreads));
    quantize_rows_kernel<T, kMode, kNorm, kGroup, kChunks><<<grid, kThreads, 0, st>>>(a);
    return launched();
}

// The most chunks of vec elements that a row of cols touches. (In 64 bits: cols goes up to 2^31 - 1.)
constexpr int64_t most_chunks(int64_t cols, int vec, RowMode mode) {
    return (cols + (mode == kTouched ? 2 * vec - 2 : vec - 1)) / vec;
}
static_assert(most_chunks(int32_t{kI32Max}, 8, kTouched) == (int64_t{1} << 28) + 1, "the longest row");

// The smallest group that holds a row: short rows then share a warp (fewer
// shuffle steps for a row, several rows' loads in flight), the shortest take a
// thread each, long ones take a block. A step stays where the next one, which
// would hold its rows too, is slower (us for 400 MB of rows at the step's
// limit, by the step / by the next):
//   whole chunks     1: 178 / 184 (bf16), 100 / 141 (f32)  2: 137 / 147  6: 141 / 235  8: 98 / 144 (f32)  16: 128 / 173
//   of bf16         32: 106 / 160   64: 105 / 166  128: 101 / 152  256: 99 / 166  512: 107 / 159  1024: 106 / 193
//                 2048: 124 / 159  4096: 105 / 132; at 4 within 3 % (f32 98 / 95)
//   touched chunks  32: 165 / 270   64: 167 / 264  128: 151 / 192  192: 144 / 191  256: 155 / 217  512: 138 / 237
//                 1024: 160 / 229  2048: 149 / 275  (4096: 182 / 177)
//   single f32      16: 203 / 278   32: 137 / 192   64: 132 / 155  128: 142 / 178  256: 103 / 148  512: 86 / 178
//                 1024: 100 / 143  2048: 87 / 201  4096: 121 / 133
template <typename T, RowMode kMode, bool kNorm>
maxsim_status launch_quantize(const QuantizeArgs& a, const HostDevice& dev, cudaStream_t st) {
    const int64_t chunks = most_chunks(a.cols, QuantizeRow<T, kMode>::C::kVec, kMode);
    if constexpr (kMode != kSingle) {
        if constexpr (kMode == kWhole) {  // measured, by single threads and by groups of 8: 3000000 x 16 bf16 32 and 133 us,
            // 3000000 x 40 bf16 82 and 145, 3000000 x 32 f32 (eight chunks) 135 and 95
            if (chunks <= 1) return launch_quantize_group<T, kMode, kNorm, 1, 1>(a, dev, st);
            if (chunks <= 2) return launch_quantize_group<T, kMode, kNorm, 1, 2>(a, dev, st);
            if (chunks <= 4) return launch_quantize_group<T, kMode, kNorm, 1, 4>(a, dev, st);
            if (chunks <= 6) return launch_quantize_group<T, kMode, kNorm, 1, 6>(a, dev, st);
            if (chunks <= 8) return launch_quantize_group<T, kMode, kNorm, 8, 1>(a, dev, st);
            if (chunks <= 16) return launch_quantize_group<T, kMode, kNorm, 8, 2>(a, dev, st);
        }
        if (chunks <= 32) return launch_quantize_group<T, kMode, kNorm, 8, 4>(a, dev, st);
        if (chunks <= 64) return launch_quantize_group<T, kMode, kNorm, 8, 8>(a, dev, st);
        if (chunks <= 128) return launch_quantize_group<T, kMode, kNorm, 32, 4>(a, dev, st);
        if constexpr (kMode == kTouched)
            if (chunks <= 192) return launch_quantize_group<T, kMode, kNorm, 32, 6>(a, dev, st);
        if (chunks <= 256) return launch_quantize_group<T, kMode, kNorm, 32, 8>(a, dev, st);
        if (chunks <= 512) return launch_quantize_group<T, kMode, kNorm, 128, 4>(a, dev, st);
        if (chunks <= 1024) return launch_quantize_group<T, kMode, kNorm, 128, 8>(a, dev, st);
        if (chunks <= 2048) return launch_quantize_group<T, kMode, kNorm, 512, 4>(a, dev, st);
        if (chunks <= 4096) return launch_quantize_group<T, kMode, kNorm, 512, 8>(a, dev, st);
    } else {  // single elements: more of them a thread
        if (chunks <= 12) return launch_quantize_group<T, kMode, kNorm, 1, 12>(a, dev, st);
        if (chunks <= 16) return launch_quantize_group<T, kMode, kNorm, 8, 2>(a, dev, st);
        if (chunks <= 32) return launch_quantize_group<T, kMode, kNorm, 8, 4>(a, dev, st);
        if (chunks <= 64) return launch_quantize_group<T, kMode, kNorm, 8, 8>(a, dev, st);
        if (chunks <= 128) return launch_quantize_group<T, kMode, kNorm, 8, 16>(a, dev, st);
        if (chunks <= 256) return launch_quantize_group<T, kMode, kNorm, 32, 8>(a, dev, st);
        if (chunks <= 512) return launch_quantize_group<T, kMode, kNorm, 32, 16>(a, dev, st);
        if (chunks <= 1024) return launch_quantize_group<T, kMode, kNorm, 32, 32>(a, dev, st);
        if (chunks <= 2048) return launch_quantize_group<T, kMode, kNorm, 128, 16>(a, dev, st);
        if (chunks <= 4096) return launch_quantize_group<T, kMode, kNorm, 512, 8>(a, dev, st);
    }
    quantize_long_rows_kernel<T, kMode, kNorm><<<grid_of(a.rows, 1, int64_t(dev.num_sms) * 4), 512, 0, st>>>(a);
    return launched();
}

template <typename T, bool kNorm>
maxsim_status launch_quantize_mode(const QuantizeArgs& a, const HostDevice& dev, cudaStream_t st) {
    constexpr int kVec = Chunk<T, true>::kVec;
    if (a.cols % kVec == 0 && a.ld_x % kVec == 0 && a.ld_q % kVec == 0 && ptr_aligned(a.x, 16) && ptr_aligned(a.q, kVec))
        return launch_quantize<T, kWhole, kNorm>(a, dev, st);
    if constexpr (sizeof(T) == 2) {
        // Measured, touched chunks and single elements: 608816 x 92 bf16 83 and 68 us, 500000 x 150 86 and 115,
        // 6847 x 2505 17 and 38, 15875 x 7518 76 and 145; f32 60000 x 2001 126 and 104.
        const uintptr_t phase = reinterpret_cast<uintptr_t>(a.x) / 2 - reinterpret_cast<uintptr_t>(a.q);
        if (a.cols >= 128 && phase % kVec == 0 && (a.rows == 1 || (a.ld_x - a.ld_q) % kVec == 0))
            return launch_quantize<T, kTouched, kNorm>(a, dev, st);
    }
    return launch_quantize<T, kSingle, kNorm>(a, dev, st);
}

template <typename T>
maxsim_status launch_quantize_any(const QuantizeArgs& a, bool normalize, const HostDevice& dev, cudaStream_t st) {
    return normalize ? launch_quantize_mode<T, true>(a, dev, st) : launch_quantize_mode<T, false>(a, dev, st);
}

// The multiplier and shift that divide 0 <= i < 2^31 by d (round-up method: with l = ceil(log2 d),
// ceil(2^(31 + l) / d) < 2^32 is exact for i < 2^31).
void set_div(DropoutArgs* a, uint32_t d) {
    if (d == 1) {
        a->div_mul = 0;
        a->div_shift = 0xffffffffu;
        return;
    }
    uint32_t l = 0;
    while ((uint64_t(1) << l) < d) ++l;
    a->div_mul = static_cast<uint32_t>(((uint64_t(1) << (31 + l)) + d - 1) / d);
    a->div_shift = l - 1;
}

template <typename T, int kX, bool kRes>
void launch_dropout_wide(const DropoutArgs& a, int64_t most, cudaStream_t st) {
    dropout_wide_kernel<T, kX, kRes><<<grid_of(a.n / 8, 256 * dropout_pieces<T, kX>(), most), 256, 0, st>>>(a);
}

template <typename T, bool kRes>
void launch_dropout_layout(DropoutArgs& a, const HostDevice& dev, cudaStream_t st) {
    constexpr int kVec = 16 / static_cast<int>(sizeof(T));
    const int64_t most = int64_t(dev.num_sms) * 8;
    const bool x16 = ptr_aligned(a.x, 16), out16 = ptr_aligned(a.y, 16) && ptr_aligned(a.residual, 16);
    const bool x_run = a.rows == 1 || a.ld_x == a.cols;
    const bool out_run = a.rows == 1 || (a.ld_y == a.cols && (!kRes || a.ld_r == a.cols));
    if (out16 && out_run && x16 && x_run) {
        launch_dropout_wide<T, kXFlat, kRes>(a, most, st);
    } else if (out16 && x16 && a.cols % 8 == 0 && a.ld_x % kVec == 0 && a.ld_y % kVec == 0 && (!kRes || a.ld_r % kVec == 0)) {
        set_div(&a, static_cast<uint32_t>(a.cols / 8));
        launch_dropout_wide<T, kXRows, kRes>(a, most, st);
    } else if (out16 && out_run && a.cols >= 8) {
        set_div(&a, static_cast<uint32_t>(a.cols));
        launch_dropout_wide<T, kXGather, kRes>(a, most, st);
    } else {
        set_div(&a, static_cast<uint32_t>(a.cols));
        const unsigned any_grid = grid_of(a.n, 8 * 256, most);
        if (a.cols >= 256) dropout_any_kernel<T, kRes, 256><<<any_grid, 256, 0, st>>>(a);
        else dropout_any_kernel<T, kRes, 0><<<any_grid, 256, 0, st>>>(a);
    }
}

template <typename T>
maxsim_status launch_dropout(DropoutArgs& a, const HostDevice& dev, cudaStream_t st) {
    if (a.residual) launch_dropout_layout<T, true>(a, dev, st);
    else launch_dropout_layout<T, false>(a, dev, st);
    return launched();
}

maxsim_status run_dropout(DropoutArgs& a, maxsim_dtype dtype, cudaStream_t st) {
    HostDevice dev;
    const maxsim_status rc = host_device(&dev);
    if (rc != MAXSIM_OK) return rc;
    if (dtype == MAXSIM_F16) return launch_dropout<__half>(a, dev, st);
    if (dtype == MAXSIM_BF16) return launch_dropout<__nv_bfloat16>(a, dev, st);
    return launch_dropout<float>(a, dev, st);
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
    const QuantizeArgs a{x, q, scale, rows, ld_x, ld_q, static_cast<int32_t>(cols)};
    if (dtype == MAXSIM_F16) return launch_quantize_any<__half>(a, normalize != 0, dev, st);
    if (dtype == MAXSIM_BF16) return launch_quantize_any<__nv_bfloat16>(a, normalize != 0, dev, st);
    return launch_quantize_any<float>(a, normalize != 0, dev, st);
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
    a.n = rows * cols;
    a.key0 = static_cast<uint32_t>(seed);
    a.key1 = static_cast<uint32_t>(seed >> 32);
    a.off0 = static_cast<uint32_t>(offset);
    a.off1 = static_cast<uint32_t>(offset >> 32);
    return run_dropout(a, dtype, static_cast<cudaStream_t>(stream));
}

maxsim_status maxsim_dropout_bwd(const void* grad, maxsim_dtype dtype, int64_t rows, int64_t cols, int64_t ld_grad,
                                 double p, uint64_t seed, uint64_t offset, void* dx, int64_t ld_dx, void* stream) {
    // the mask is the forward's, drawn again: the same map without a residual
    return maxsim_dropout_fwd(grad, dtype, rows, cols, ld_grad, nullptr, 0, p, seed, offset, dx, ld_dx, stream);
}

}  // extern "C"
