// Host side of the log probabilities and their gradient (include/maxsim.h):
// argument validation and the launches on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "maxsim.h"
#include "host_util.h"
#include "logprobs_kernels.cuh"

namespace maxsim {
namespace {

constexpr int kMaxTargets = 256;
constexpr double kLog2E = 1.4426950408889634;

template <typename T, bool kMask, bool kTop, int kThreads>
maxsim_status launch_block(const LogprobsArgs& a, int blocks, const HostDevice& dev, cudaStream_t st) {
    auto kern = logprobs_block_kernel<T, kMask, kTop, kThreads>;
    if (blocks > 8) {  // clusters of 16 are asked for by name
        static std::atomic<uint64_t> prepared{0};
        const uint64_t bit = uint64_t(1) << dev.index;
        if (!(prepared.load(std::memory_order_acquire) & bit)) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return MAXSIM_ERR_CUDA;
            prepared.fetch_or(bit, std::memory_order_release);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows * blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kTop && blocks > 1 ? static_cast<size_t>(blocks) * a.k * 8 : 0;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(blocks);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kern, a, blocks) != cudaSuccess) {
        cudaGetLastError();
        return MAXSIM_ERR_CUDA;
    }
    return MAXSIM_OK;
}

template <typename T, bool kMask, bool kTop>
maxsim_status launch_fwd(const LogprobsArgs& a, const HostDevice& dev, cudaStream_t st) {
    const int64_t pieces = (a.n * static_cast<int64_t>(sizeof(T)) + 15) / 16;
    const unsigned warps = static_cast<unsigned>((a.rows + 7) / 8);
    // Short rows take a warp each. Their strongest columns by ranks or one after another (us for 16,384 f32 rows
    // without any, by ranks, and for each listed one: 64 columns 8, 20, 1.5; 128: 8, 50, 1.6; 250 bf16: 11, 176, 1.5). A
    // warp alone takes 0.3 us for each one, so that few rows are ranked sooner, or take a block (100 x 500 f32
    // with 64 listed 19 and 8 us, with 8 5.4 and 5.7; 3000 x 2000 bf16 with 64 39 and 29, with 20 16 and 18).
    const bool few = a.rows <= int64_t(dev.num_sms) * 8;
    if constexpr (kTop) {
        if (a.n <= kRankColumns && (a.n * a.n <= int64_t(600) * a.k || (few && a.k > 16))) {
            logprobs_warp_kernel<T, kMask, 2><<<warps, 256, 0, st>>>(a);
            return launched();
        }
    }
    const bool block = few ? a.k > 8 && pieces > 32 : a.k >= 32 && a.rows <= int64_t(dev.num_sms) * 32 && pieces > 64;
    if (pieces <= 256 && !block) {
        logprobs_warp_kernel<T, kMask, kTop ? 1 : 0><<<warps, 256, 0, st>>>(a);
        return launched();
    }
    // few rows: the blocks of a cluster share one
    int blocks = 1;
    while (blocks < 16 && a.rows * blocks * 2 <= int64_t(dev.num_sms) * 4 && pieces / (blocks * 2) >= 512) blocks *= 2;
    // Threads of a block, by the GPU times with 128 and 256 (us). Where all blocks run at once, more threads pay for long
    // shares: 1 x 300000 f32 5.9 and 4.7 (4,687 pieces a block), 600 x 1000000 bf16 239 and 185, but 150 x 65536 bf16 6.5
    // and 7.7 (2,048 pieces). Where they take turns, more blocks do, until many columns are listed: 4096 x 131072 bf16
    // without any 157 and 162, with 5 186 and 209, with 20 203 and 217, with 64 274 and 246; 5000 x 131072 f16 with 32
    // 271 and 278, with 40 287 and 282; 8192 x 32768 bf16 with 64 157 and 185 (4,096 pieces). (f32 rows without any lose
    // by it: 700 x 400000 183 and 158, 4096 x 32768 79 and 81.)
    const bool at_once = a.rows * blocks <= int64_t(dev.num_sms) * 4;
    if (at_once ? pieces / blocks <= 4096 : pieces <= 8192 || a.k < 40) return launch_block<T, kMask, kTop, 128>(a, blocks, dev, st);
    return launch_block<T, kMask, kTop, 256>(a, blocks, dev, st);
}

template <typename T>
maxsim_status run_fwd(const LogprobsArgs& a, const HostDevice& dev, cudaStream_t st) {
    if (a.mask) return a.k ? launch_fwd<T, true, true>(a, dev, st) : launch_fwd<T, true, false>(a, dev, st);
    return a.k ? launch_fwd<T, false, true>(a, dev, st) : launch_fwd<T, false, false>(a, dev, st);
}

template <typename T, bool kMask>
maxsim_status launch_bwd(const LogprobsBwdArgs& a, const HostDevice& dev, cudaStream_t st) {
    // a row off its 16-byte boundary touches one piece more
    const int64_t pieces = (a.n * static_cast<int64_t>(sizeof(T)) + 15) / 16 + 1;
    const bool same = ((reinterpret_cast<uintptr_t>(a.x) - reinterpret_cast<uintptr_t>(a.dx)) & 15) == 0 &&
                      (a.rows == 1 || (a.ld - a.ld_dx) * static_cast<int64_t>(sizeof(T)) % 16 == 0);
    // A warp's run: long ones read the row's numbers less often, but every SM wants warps.
    const int64_t least = 32 * BwdCfg::kPieces;
    int64_t run = 12 * least;
    while (run > least && a.rows * ((pieces + run - 1) / run) < int64_t(dev.num_sms) * 64) run /= 2;
    run = (run + least - 1) / least * least;
    const int64_t runs = (pieces + run - 1) / run, items = a.rows * runs;
    if ((items + 7) / 8 > kI32Max) return MAXSIM_ERR_UNSUPPORTED;
    const unsigned grid = static_cast<unsigned>((items + 7) / 8);
    if (same) logprobs_bwd_kernel<T, kMask, false><<<grid, 256, 0, st>>>(a, static_cast<int32_t>(run), runs, items);
    else logprobs_bwd_kernel<T, kMask, true><<<grid, 256, 0, st>>>(a, static_cast<int32_t>(run), runs, items);
    return launched();
}

template <typename T>
maxsim_status run_bwd(const LogprobsBwdArgs& a, const HostDevice& dev, cudaStream_t st) {
    return a.mask ? launch_bwd<T, true>(a, dev, st) : launch_bwd<T, false>(a, dev, st);
}

// What both directions ask of the rows, the given columns and the mask.
maxsim_status check_rows(const void* x, maxsim_dtype dtype, int64_t rows, int64_t n, int64_t ld, const int64_t* targets, int64_t T,
                         const uint8_t* mask, int64_t ld_mask, double scale, int64_t k) {
    if (!any_dtype(dtype) || rows < 0 || n < 1 || T < 0 || k < 0 || !(scale > 0.0) || !std::isfinite(static_cast<float>(scale * kLog2E)))
        return MAXSIM_ERR_INVALID_ARG;
    if (static_cast<float>(scale) == 0.f || k > n) return MAXSIM_ERR_INVALID_ARG;
    if (!rows_fit(rows, n, ld) || (mask && ld_mask != 0 && !rows_fit(rows, n, ld_mask))) return MAXSIM_ERR_INVALID_ARG;
    if (rows > kI32Max / 16 || n > kI32Max - 1024 || T > kMaxTargets || k > kLogprobsMaxTop) return MAXSIM_ERR_UNSUPPORTED;
    if (rows == 0) return MAXSIM_OK;
    if (!x || !ptr_aligned(x, elem_bytes(dtype)) || (T > 0 && (!targets || !ptr_aligned(targets, 8)))) return MAXSIM_ERR_INVALID_ARG;
    return MAXSIM_OK;
}

// Whether two [rows, n] operands may share elements: their ranges meet, and they
// are not columns side by side of rows that are equally far apart.
bool rows_overlap(const void* x, int64_t ld_x, const void* y, int64_t ld_y, int64_t rows, int64_t n, int64_t bytes) {
    const uintptr_t px = reinterpret_cast<uintptr_t>(x), py = reinterpret_cast<uintptr_t>(y);
    const uintptr_t end_x = px + static_cast<uintptr_t>(((rows - 1) * ld_x + n) * bytes), end_y = py + static_cast<uintptr_t>(((rows - 1) * ld_y + n) * bytes);
    if (px >= end_y || py >= end_x) return false;
    if (rows == 1 || ld_x != ld_y) return true;
    const uintptr_t row = static_cast<uintptr_t>(ld_x * bytes), off = (py > px ? py - px : px - py) % row, wide = static_cast<uintptr_t>(n * bytes);
    return off < wide || row - off < wide;
}

}  // namespace
}  // namespace maxsim

using namespace maxsim;

extern "C" {

maxsim_status maxsim_logprobs_fwd(const void* logits, maxsim_dtype dtype, int64_t rows, int64_t n, int64_t ld,
                                  const int64_t* targets, int64_t T, const uint8_t* mask, int64_t ld_mask, double scale,
                                  int64_t k, float* logprob, float* entropy, int32_t* top_idx, float* top_logprob,
                                  float* stats, void* stream) {
    const maxsim_status ok = check_rows(logits, dtype, rows, n, ld, targets, T, mask, ld_mask, scale, k);
    if (ok != MAXSIM_OK || rows == 0) return ok;
    if ((T > 0 && !logprob) || !entropy || !stats || (k > 0 && (!top_idx || !top_logprob))) return MAXSIM_ERR_INVALID_ARG;
    if (!ptr_aligned(logprob, 4) || !ptr_aligned(entropy, 4) || !ptr_aligned(stats, 8) || !ptr_aligned(top_idx, 4) || !ptr_aligned(top_logprob, 4))
        return MAXSIM_ERR_INVALID_ARG;
    HostDevice dev;
    const maxsim_status rc = host_device(&dev);
    if (rc != MAXSIM_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const LogprobsArgs a{logits, targets, mask, rows, n, ld, ld_mask, static_cast<int32_t>(T), static_cast<int32_t>(k),
                         static_cast<float>(scale), static_cast<float>(scale * kLog2E), logprob, entropy, top_idx, top_logprob, stats, dev.status};
    if (dtype == MAXSIM_F16) return run_fwd<__half>(a, dev, st);
    if (dtype == MAXSIM_BF16) return run_fwd<__nv_bfloat16>(a, dev, st);
    return run_fwd<float>(a, dev, st);
}

maxsim_status maxsim_logprobs_bwd(const void* logits, maxsim_dtype dtype, int64_t rows, int64_t n, int64_t ld,
                                  const int64_t* targets, int64_t T, const uint8_t* mask, int64_t ld_mask, double scale,
                                  const float* stats, const float* entropy, const float* grad_logprob,
                                  const float* grad_entropy, const int32_t* top_idx, const float* grad_top, int64_t k,
                                  void* dx, int64_t ld_dx, void* stream) {
    if (!grad_top) {  // neither is read
        k = 0;
        top_idx = nullptr;
    }
    const maxsim_status ok = check_rows(logits, dtype, rows, n, ld, targets, T, mask, ld_mask, scale, k);
    if (ok != MAXSIM_OK) return ok;
    if (!rows_fit(rows, n, ld_dx)) return MAXSIM_ERR_INVALID_ARG;
    if (rows == 0) return MAXSIM_OK;
    if (!dx || !ptr_aligned(dx, elem_bytes(dtype)) || !stats || !ptr_aligned(stats, 8) || (grad_entropy && !entropy) ||
        (grad_top && !top_idx))
        return MAXSIM_ERR_INVALID_ARG;
    // every warp of a row reads the given columns' logits, those of other warps' runs among them
    if (rows_overlap(logits, ld, dx, ld_dx, rows, n, elem_bytes(dtype))) return MAXSIM_ERR_INVALID_ARG;
    if (!ptr_aligned(entropy, 4) || !ptr_aligned(grad_logprob, 4) || !ptr_aligned(grad_entropy, 4) || !ptr_aligned(top_idx, 4) ||
        !ptr_aligned(grad_top, 4))
        return MAXSIM_ERR_INVALID_ARG;
    HostDevice dev;
    const maxsim_status rc = host_device(&dev);
    if (rc != MAXSIM_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const LogprobsBwdArgs a{logits, targets, mask, rows, n, ld, ld_mask, ld_dx, static_cast<int32_t>(T), static_cast<int32_t>(k),
                            static_cast<float>(scale), static_cast<float>(scale * kLog2E), stats, entropy, grad_logprob, grad_entropy,
                            top_idx, grad_top, dx, dev.status};
    if (dtype == MAXSIM_F16) return run_bwd<__half>(a, dev, st);
    if (dtype == MAXSIM_BF16) return run_bwd<__nv_bfloat16>(a, dev, st);
    return run_bwd<float>(a, dev, st);
}

}  // extern "C"
