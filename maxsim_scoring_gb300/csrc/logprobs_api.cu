// Host side of the log probabilities and their gradient (include/maxsim.h):
// argument validation and the launches on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
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
    const int64_t most = std::max<int64_t>(1, int64_t(dev.num_sms) * (2048 / kThreads) / blocks);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min(a.rows, most) * blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(blocks);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, logprobs_block_kernel<T, kMask, kTop, kThreads>, a, blocks) != cudaSuccess) {
        cudaGetLastError();
        return MAXSIM_ERR_CUDA;
    }
    return MAXSIM_OK;
}

template <typename T, bool kMask, bool kTop>
maxsim_status launch_fwd(const LogprobsArgs& a, const HostDevice& dev, cudaStream_t st) {
    const int64_t pieces = (a.n * static_cast<int64_t>(sizeof(T)) + 15) / 16;
    if (!kTop && pieces <= 256) {
        logprobs_warp_kernel<T, kMask><<<grid_of(a.rows, 8, int64_t(dev.num_sms) * 8), 256, 0, st>>>(a);
        return launched();
    }
    int blocks = 1;
    while (blocks < 8 && a.rows * blocks * 2 <= int64_t(dev.num_sms) * 4 && pieces / (blocks * 2) >= 1024) blocks *= 2;
    if (pieces / blocks <= 1024) return launch_block<T, kMask, kTop, 128>(a, blocks, dev, st);
    return launch_block<T, kMask, kTop, 512>(a, blocks, dev, st);
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
    if (pieces <= 128) {
        logprobs_bwd_kernel<T, kMask, 32, 4><<<grid_of(a.rows, 8, int64_t(1) << 30), 256, 0, st>>>(a, 1, a.rows);
        return launched();
    }
    const int64_t runs = (pieces + 1023) / 1024, items = a.rows * runs;
    logprobs_bwd_kernel<T, kMask, 256, 4><<<grid_of(items, 1, int64_t(1) << 30), 256, 0, st>>>(a, runs, items);
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
    if (static_cast<float>(scale * kLog2E) == 0.f || k > n) return MAXSIM_ERR_INVALID_ARG;
    if (!rows_fit(rows, n, ld) || (mask && ld_mask != 0 && !rows_fit(rows, n, ld_mask))) return MAXSIM_ERR_INVALID_ARG;
    if (rows > kI32Max || n > kI32Max - 1024 || T > kMaxTargets || k > kLogprobsMaxTop) return MAXSIM_ERR_UNSUPPORTED;
    if (rows == 0) return MAXSIM_OK;
    if (!x || !ptr_aligned(x, elem_bytes(dtype)) || (T > 0 && (!targets || !ptr_aligned(targets, 8)))) return MAXSIM_ERR_INVALID_ARG;
    return MAXSIM_OK;
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
    if (!ptr_aligned(logprob, 4) || !ptr_aligned(entropy, 4) || !ptr_aligned(stats, 4) || !ptr_aligned(top_idx, 4) || !ptr_aligned(top_logprob, 4))
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
    const maxsim_status ok = check_rows(logits, dtype, rows, n, ld, targets, T, mask, ld_mask, scale, k);
    if (ok != MAXSIM_OK) return ok;
    if (!rows_fit(rows, n, ld_dx)) return MAXSIM_ERR_INVALID_ARG;
    if (rows == 0) return MAXSIM_OK;
    if (!dx || !ptr_aligned(dx, elem_bytes(dtype)) || !stats || !ptr_aligned(stats, 4) || (grad_entropy && !entropy) ||
        (grad_top && !top_idx))
        return MAXSIM_ERR_INVALID_ARG;
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
