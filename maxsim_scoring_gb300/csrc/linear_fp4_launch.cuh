// Launches of the 4-bit linear, per output type (linear_fp4_f16.cu,
// linear_fp4_bf16.cu, linear_fp4_f32.cu, compiled side by side).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "maxsim.h"
#include "host_util.h"
#include "linear_fp4.cuh"

namespace maxsim {

// [rows, bytes] codes, rows ld bytes apart, in boxes of 128 bytes x box_rows.
inline bool encode_codes(EncodeTiledFn encode, CUtensorMap* map, const void* base, int64_t bytes, int64_t rows, int64_t ld, uint32_t box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(bytes), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(rows > 1 ? ld : bytes)};
    const cuuint32_t box[2] = {128, box_rows}, estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles [row tiles, words] of 512 bytes (256 16-bit values), box_words x box_tiles of them a box.
inline bool encode_scales(EncodeTiledFn encode, CUtensorMap* map, const void* base, int64_t words, int64_t rows, uint32_t box_words, uint32_t box_tiles) {
    const cuuint64_t dims[3] = {256, static_cast<cuuint64_t>(words), static_cast<cuuint64_t>((rows + 127) / 128)};
    const cuuint64_t strides[2] = {512, static_cast<cuuint64_t>(words) * 512};
    const cuuint32_t box[3] = {256, box_words, box_tiles}, estr[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int kTN, bool kSwap, bool kRows16>
maxsim_status launch_fp4_kernel(const LinearFp4Plan& p, const LinearFp4Args& l, int block, const HostDevice& dev, cudaStream_t st) {
    using C = Fp4Cfg<kTN>;
    auto kern = linear_fp4_kernel<T, kTN, kSwap, kRows16>;
    constexpr size_t kSmem = fp4_smem_bytes<kTN>();
    static_assert(kSmem <= kSmemBudget, "shared memory of one SM");
    static_assert(kTN != 64 || (kFp4MaxSplits - 1) * kTN * 128 * 4 <= C::kStages * (C::kA + C::kB), "the splits' sums lie in the stages");
    static std::atomic<uint64_t> prepared{0};  // devices whose shared-memory limit is raised
    const uint64_t bit = uint64_t(1) << dev.index;
    if (!(prepared.load(std::memory_order_acquire) & bit)) {
        // the register split adds up only if every thread is launched with kFp4Regs
        cudaFuncAttributes fa{};
        if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return MAXSIM_ERR_CUDA;
        if (fa.numRegs < kFp4Regs) return MAXSIM_ERR_UNSUPPORTED;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)) != cudaSuccess)
            return MAXSIM_ERR_CUDA;
        prepared.fetch_or(bit, std::memory_order_release);
    }
    LinearFp4TileArgs a{};
    a.l = l;
    a.items = p.tiles;
    a.rows_a = kSwap ? l.N : l.M;
    a.rows_b = kSwap ? l.M : l.N;
    a.tiles_b = static_cast<int32_t>(p.tiles_b);
    a.kb = p.kb;
    a.splits = p.splits;
    a.kb_split = p.kb_split;
    a.block = block;
    a.prefetch = p.tiles_b >= 4;
    a.status = dev.status;
    a.timeout_ns = kTimeoutNs;
    CUtensorMap ta, tb, fa, fb;
    const uint32_t words = block == 16 ? 4 : 2;
    if (!encode_codes(dev.encode, &ta, kSwap ? l.w : l.x, l.K / 2, a.rows_a, kSwap ? l.ld_w : l.ld_x, 128) ||
        !encode_codes(dev.encode, &tb, kSwap ? l.x : l.w, l.K / 2, a.rows_b, kSwap ? l.ld_x : l.ld_w, C::kBRows) ||
        !encode_scales(dev.encode, &fa, kSwap ? l.w_block : l.x_block, l.words, a.rows_a, words, 1) ||
        !encode_scales(dev.encode, &fb, kSwap ? l.x_block : l.w_block, l.words, a.rows_b, words, C::kBTiles))
        return MAXSIM_ERR_CUDA;
    CUtensorMap tout = ta;  // used by 16-bit outputs that are stored by TMA alone
    if constexpr (sizeof(T) == 2 && kRows16 && !kSwap) {
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(l.N), static_cast<cuuint64_t>(l.M)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(l.ld_out) * 2};
        const cuuint32_t box[2] = {kTN == 64 ? 32u : 64u, 32}, estr[2] = {1, 1};
        if (dev.encode(&tout, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, l.out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       kTN == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return MAXSIM_ERR_CUDA;
    }
    const unsigned cluster = 2u * static_cast<unsigned>(p.splits);
    const int64_t most = p.splits > 1 ? p.tiles : std::max(1, dev.num_sms / 2);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(a.items, most)) * cluster);
    cfg.blockDim = dim3(kFp4Threads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, ta, tb, fa, fb, tout, a) != cudaSuccess) {
        cudaGetLastError();
        return MAXSIM_ERR_CUDA;
    }
    return MAXSIM_OK;
}

template <typename T, int kTN>
maxsim_status launch_fp4_tile(const LinearFp4Plan& p, const LinearFp4Args& l, int block, const HostDevice& dev, cudaStream_t st) {
    if (p.swap) return launch_fp4_kernel<T, kTN, true, false>(p, l, block, dev, st);
    // 16-bit outputs leave by TMA, which wants strides below 2^40 bytes and
    // writes an odd row's last element with the one behind it
    bool rows16 = ptr_aligned(l.out, 16) && l.ld_out * static_cast<int64_t>(sizeof(T)) % 16 == 0;
    if (sizeof(T) == 2) rows16 = rows16 && l.N % 8 == 0 && l.ld_out < (int64_t(1) << 38);
    return rows16 ? launch_fp4_kernel<T, kTN, false, true>(p, l, block, dev, st)
                  : launch_fp4_kernel<T, kTN, false, false>(p, l, block, dev, st);
}

template <typename T>
maxsim_status run_linear_fp4(const LinearFp4Plan& p, const LinearFp4Args& l, int block, const HostDevice& dev, cudaStream_t st) {
    if (l.K == 0) {
        linear_fp4_bias_kernel<T><<<grid_of(static_cast<int64_t>(l.M) * l.N, 256, int64_t(dev.num_sms) * 8), 256, 0, st>>>(l);
        return launched();
    }
    if (p.tn == 256) return launch_fp4_tile<T, 256>(p, l, block, dev, st);
    if (p.tn == 128) return launch_fp4_tile<T, 128>(p, l, block, dev, st);
    return launch_fp4_tile<T, 64>(p, l, block, dev, st);
}

}  // namespace maxsim
