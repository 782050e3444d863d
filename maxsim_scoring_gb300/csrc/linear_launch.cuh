// Launches of the INT8 linear, per output type (linear_f16.cu, linear_bf16.cu,
// linear_f32.cu, linear_sums.cu for the sums of slices: most of the library's
// kernels, compiled side by side).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "maxsim.h"
#include "host_util.h"
#include "linear_int8.cuh"

namespace maxsim {

struct LinearPlan {
    bool few = false;
    bool swap = false;   // A is w, B is x
    bool keep_b = false; // B stays in shared memory
    int tn = 256;
    int64_t tiles = 0, tiles_b = 0;
    int32_t kb = 0, slices = 1, kb_slice = 0;
    int64_t k_pad = 0;
    size_t off_x = 0, off_w = 0, off_b = 0, off_partial = 0, bytes = 0;
};

// Rows of K elements, ld bytes apart, in boxes of box_bytes (128 or 64) x box_rows, swizzled as wide.
inline bool encode_k_rows(EncodeTiledFn encode, CUtensorMap* map, CUtensorMapDataType type, int elem, const void* base,
                   int64_t K, int64_t rows, int64_t ld, uint32_t box_rows, uint32_t box_bytes = 128) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
    const cuuint32_t box[2] = {box_bytes / static_cast<cuuint32_t>(elem), box_rows}, estr[2] = {1, 1};
    return encode(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch that may begin before the kernel in front of it has ended (the
// kernel waits for it where it reads its results), in clusters of `cluster`.
template <typename... Params, typename... Args>
maxsim_status launch_after(void (*kern)(Params...), unsigned grid, unsigned threads, size_t smem, unsigned cluster,
                           cudaStream_t st, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
        cudaGetLastError();
        return MAXSIM_ERR_CUDA;
    }
    return MAXSIM_OK;
}

template <typename T, int kTiles>
maxsim_status launch_few(const LinearArgs& a, bool whole, cudaStream_t st) {
    const int64_t chunks = (static_cast<int64_t>(a.K) + 63) / 64;
    const int64_t blocks = (static_cast<int64_t>(a.N) + 15) / 16 * ((static_cast<int64_t>(a.M) + 8 * kTiles - 1) / (8 * kTiles));
    int64_t warps = std::min<int64_t>(kFewWarps, std::max<int64_t>(chunks, 1));
    // Fewer warps with longer runs of K once there are enough blocks: a block
    // starts and joins its warps' sums once. Measured with at most 4,096 and
    // 2,048 warps in all: 1 x 4096 x 16384 14.4 and 18.3 us, but
    // 32 x 4096 x 4096 10.2 and 8.3 us (more registers a warp).
    const int64_t most_warps = kTiles == 1 ? 4096 : 2048;
    while (warps > 4 && blocks * warps > most_warps) warps = (warps + 1) / 2;
    const unsigned threads = 32u * static_cast<unsigned>(warps);
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.N) + 15) / 16),
                    static_cast<unsigned>((static_cast<int64_t>(a.M) + 8 * kTiles - 1) / (8 * kTiles)));
    if (whole) linear_few_kernel<T, kTiles, true><<<grid, threads, 0, st>>>(a);
    else linear_few_kernel<T, kTiles, false><<<grid, threads, 0, st>>>(a);
    return launched();
}

template <typename T, int kTN, bool kSwap, bool kKeepB, bool kRows16, bool kParts>
maxsim_status launch_tile_kernel(const LinearPlan& p, const LinearArgs& l, const __half* b16, bool a_prepared, int32_t* partial,
                          const HostDevice& dev, cudaStream_t st) {
    auto kern = linear_tile_kernel<T, kTN, kSwap, kKeepB, kRows16, kParts>;
    constexpr size_t kSmem = tile_smem_bytes<kTN, kKeepB>();
    static_assert(kSmem <= kSmemBudget, "shared memory of one SM");
    static std::atomic<uint64_t> prepared{0};  // devices whose shared-memory limit is raised
    const uint64_t bit = uint64_t(1) << dev.index;
    if (!(prepared.load(std::memory_order_acquire) & bit)) {
        // the register split adds up only if every thread is launched with kTileRegs
        cudaFuncAttributes fa{};
        if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return MAXSIM_ERR_CUDA;
        if (fa.numRegs < kTileRegs) return MAXSIM_ERR_UNSUPPORTED;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)) != cudaSuccess)
            return MAXSIM_ERR_CUDA;
        prepared.fetch_or(bit, std::memory_order_release);
    }
    TileArgs a{};
    a.l = l;
    a.partial = partial;
    a.items = p.tiles * p.slices;
    a.rows_a = kSwap ? l.N : l.M;
    a.rows_b = kSwap ? l.M : l.N;
    a.tiles_b = static_cast<int32_t>(p.tiles_b);
    a.slices = p.slices;
    a.kb = p.kb;
    a.kb_slice = p.kb_slice;
    const int32_t parts = (p.kb_slice + kExactBlocks - 1) / kExactBlocks;
    a.kb_part = (p.kb_slice + parts - 1) / parts;
    a.a_prepared = a_prepared;
    a.status = dev.status;
    a.timeout_ns = kTimeoutNs;
    CUtensorMap ta, tb;
    if (!encode_k_rows(dev.encode, &ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kSwap ? l.w : l.x, l.K, a.rows_a,
                       kSwap ? l.ld_w : l.ld_x, 128) ||
        !encode_k_rows(dev.encode, &tb, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, b16, p.k_pad, a.rows_b, p.k_pad * 2,
                       TileCfg<kTN, kKeepB>::kBRows))
        return MAXSIM_ERR_CUDA;
    CUtensorMap tout = tb;  // used by 16-bit outputs that are stored by TMA alone
    if constexpr (sizeof(T) == 2 && kRows16 && !kSwap) {
        if (!encode_k_rows(dev.encode, &tout, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, l.out, l.N, l.M,
                                            l.ld_out * 2, 32, kTN == 64 ? 64 : 128))
            return MAXSIM_ERR_CUDA;
    }
    return launch_after(kern, static_cast<unsigned>(2 * std::min<int64_t>(a.items, std::max(1, dev.num_sms / 2))), kTileThreads,
                        kSmem, 2, st, ta, tb, tout, a);
}

template <typename T, int kTN, bool kSwap, bool kKeepB, bool kRows16>
maxsim_status launch_tile_rows(const LinearPlan& p, const LinearArgs& l, const __half* b16, bool a_prepared, int32_t* partial,
                               const HostDevice& dev, cudaStream_t st) {
    if constexpr (sizeof(T) == 4 && kTN <= 128 && !(kKeepB && TileCfg<kTN, kKeepB>::kStagesB <= kExactBlocks)) {
        if (parts_needed(p.kb_slice))
            return launch_tile_kernel<T, kTN, kSwap, kKeepB, kRows16, true>(p, l, b16, a_prepared, partial, dev, st);
    }
    return launch_tile_kernel<T, kTN, kSwap, kKeepB, kRows16, false>(p, l, b16, a_prepared, partial, dev, st);
}

template <typename T, int kTN, bool kSwap, bool kKeepB>
maxsim_status launch_tile(const LinearPlan& p, const LinearArgs& l, const __half* b16, bool a_prepared, int32_t* partial,
                          const HostDevice& dev, cudaStream_t st) {
    if constexpr (!kSwap) {  // swapped, a store is one channel per lane in any case
        // 16-bit outputs leave by TMA, which wants strides below 2^40 bytes and
        // writes an odd row's last element with the one behind it
        bool rows16 = std::is_same_v<T, int32_t> ? l.N % 4 == 0 : ptr_aligned(l.out, 16) && l.ld_out * static_cast<int64_t>(sizeof(T)) % 16 == 0;
        if (sizeof(T) == 2) rows16 = rows16 && l.N % 8 == 0 && l.ld_out < (int64_t(1) << 38);
        if (!rows16) return launch_tile_rows<T, kTN, kSwap, kKeepB, false>(p, l, b16, a_prepared, partial, dev, st);
    }
    return launch_tile_rows<T, kTN, kSwap, kKeepB, true>(p, l, b16, a_prepared, partial, dev, st);
}

template <typename T, bool kSwap>
maxsim_status launch_tile_width(const LinearPlan& p, const LinearArgs& l, const __half* b16, bool a_prepared, int32_t* partial,
                                const HostDevice& dev, cudaStream_t st) {
    if constexpr (!kSwap && !std::is_same_v<T, int32_t>) {
        if (p.keep_b && p.tn == 128) return launch_tile<T, 128, false, true>(p, l, b16, a_prepared, partial, dev, st);
        if (p.keep_b) return launch_tile<T, 64, false, true>(p, l, b16, a_prepared, partial, dev, st);
    }
    if constexpr (!std::is_same_v<T, int32_t>) {
        if (p.tn == 256) return launch_tile<T, 256, kSwap, false>(p, l, b16, a_prepared, partial, dev, st);
    }
    if (p.tn == 128) return launch_tile<T, 128, kSwap, false>(p, l, b16, a_prepared, partial, dev, st);
    return launch_tile<T, 64, kSwap, false>(p, l, b16, a_prepared, partial, dev, st);
}

// The tile kernel for outputs of T, or for the integer sums of slices (int32_t).
template <typename T>
maxsim_status launch_tiles(const LinearPlan& p, const LinearArgs& l, const __half* b16, bool a_prepared, int32_t* partial,
                           const HostDevice& dev, cudaStream_t st) {
    return p.swap ? launch_tile_width<T, true>(p, l, b16, a_prepared, partial, dev, st)
                  : launch_tile_width<T, false>(p, l, b16, a_prepared, partial, dev, st);
}

extern template maxsim_status launch_tiles<int32_t>(const LinearPlan&, const LinearArgs&, const __half*, bool, int32_t*,
                                                    const HostDevice&, cudaStream_t);  // linear_sums.cu

template <typename T>
maxsim_status run_linear(const LinearPlan& p, LinearArgs l, bool x_direct, bool w_direct, uint8_t* ws,
                         const HostDevice& dev, cudaStream_t st) {
    const int64_t most = int64_t(dev.num_sms) * 8;
    const unsigned join_grid = grid_of(static_cast<int64_t>(l.M) * l.N, 256, most);
    if (l.K == 0) {  // no products: the bias
        linear_join_kernel<T><<<join_grid, 256, 0, st>>>(l, nullptr, 0);
        return launched();
    }
    if (p.few) {
        const bool whole = x_direct && w_direct;
        if (l.M <= 8) return launch_few<T, 1>(l, whole, st);
        if (l.M <= 16) return launch_few<T, 2>(l, whole, st);
        return launch_few<T, 4>(l, whole, st);
    }
    const int32_t k_pad = static_cast<int32_t>(p.k_pad);
    const __half* b16 = reinterpret_cast<const __half*>(ws + p.off_b);
    const bool copy_x = !x_direct && !p.swap, copy_w = !w_direct && p.swap;
    PrepArgs prep{};
    prep.K = l.K;
    prep.k_pad = k_pad;
    prep.widen = {p.swap ? l.x : l.w, ws + p.off_b, p.swap ? l.M : l.N, p.swap ? l.ld_x : l.ld_w,
                  p.swap ? x_direct : w_direct};
    if (copy_x) prep.copy = {l.x, ws + p.off_x, l.M, l.ld_x, 0};
    if (copy_w) prep.copy = {l.w, ws + p.off_w, l.N, l.ld_w, 0};
    linear_prep_kernel<<<grid_of((prep.widen.rows + prep.copy.rows) * (k_pad / 16), 256, most), 256, 0, st>>>(prep);
    if (copy_x) {
        l.x = reinterpret_cast<const int8_t*>(ws + p.off_x);
        l.ld_x = k_pad;
    }
    if (copy_w) {
        l.w = reinterpret_cast<const int8_t*>(ws + p.off_w);
        l.ld_w = k_pad;
    }
    l.K = k_pad;  // an operand read where it is has K % 16 == 0 already; repacked tails are zero
    maxsim_status rc = launched();
    if (rc != MAXSIM_OK) return rc;
    int32_t* partial = reinterpret_cast<int32_t*>(ws + p.off_partial);
    const bool prepared = copy_x || copy_w;
    if (p.slices == 1) return launch_tiles<T>(p, l, b16, prepared, partial, dev, st);
    rc = launch_tiles<int32_t>(p, l, b16, prepared, partial, dev, st);
    if (rc != MAXSIM_OK) return rc;
    return launch_after(linear_join_kernel<T>, join_grid, 256, 0, 1, st, l, const_cast<const int32_t*>(partial), p.slices);
}

}  // namespace maxsim
