// Host side of the token head's entry points (include/maxsim.h): argument
// validation and the launches on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "maxsim.h"
#include "host_util.h"
#include "head_kernels.cuh"
#include "linear_int8.cuh"

namespace maxsim {
namespace {

constexpr int64_t kI32Max = 2147483647;
constexpr int64_t kLinearMaxK = 131071;             // 131071 * 128 * 128 < 2^31
constexpr int64_t kLinearMaxRows = 2147483647 - 1023;  // a tile past the last row still has 32-bit coordinates

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

template <typename T, bool kWide, bool kNorm, int kGroup, int kChunks>
maxsim_status launch_quantize_group(const QuantizeArgs& a, const HostDevice& dev, cudaStream_t st) {
    constexpr int kThreads = quantize_threads(kGroup);
    const unsigned grid = grid_of(a.rows, kThreads / kGroup, int64_t(dev.num_sms) * (2048 / kThreads));
    quantize_rows_kernel<T, kWide, kNorm, kGroup, kChunks><<<grid, kThreads, 0, st>>>(a);
    return launched();
}

// The smallest group that holds a row: short rows then share a warp (fewer
// shuffle steps for a row, several rows' loads in flight), long ones take a
// block.
template <typename T, bool kWide, bool kNorm>
maxsim_status launch_quantize(const QuantizeArgs& a, const HostDevice& dev, cudaStream_t st) {
    const int64_t chunks = (a.cols + Chunk<T, kWide>::kVec - 1) / Chunk<T, kWide>::kVec;
    if constexpr (kWide) {
        if (chunks <= 8) return launch_quantize_group<T, kWide, kNorm, 8, 1>(a, dev, st);
        if (chunks <= 16) return launch_quantize_group<T, kWide, kNorm, 8, 2>(a, dev, st);
        if (chunks <= 32) return launch_quantize_group<T, kWide, kNorm, 8, 4>(a, dev, st);
        if (chunks <= 64) return launch_quantize_group<T, kWide, kNorm, 8, 8>(a, dev, st);
        if (chunks <= 128) return launch_quantize_group<T, kWide, kNorm, 32, 4>(a, dev, st);
        if (chunks <= 256) return launch_quantize_group<T, kWide, kNorm, 32, 8>(a, dev, st);
        if (chunks <= 512) return launch_quantize_group<T, kWide, kNorm, 128, 4>(a, dev, st);
        if (chunks <= 1024) return launch_quantize_group<T, kWide, kNorm, 128, 8>(a, dev, st);
        if (chunks <= 2048) return launch_quantize_group<T, kWide, kNorm, 512, 4>(a, dev, st);
        if (chunks <= 4096) return launch_quantize_group<T, kWide, kNorm, 512, 8>(a, dev, st);
    } else {  // single elements: more of them a thread
        if (chunks <= kNarrow) {
            quantize_narrow_rows_kernel<T, kNorm><<<grid_of(a.rows, 128, int64_t(dev.num_sms) * 16), 128, 0, st>>>(a);
            return launched();
        }
        if (chunks <= 16) return launch_quantize_group<T, kWide, kNorm, 8, 2>(a, dev, st);
        if (chunks <= 32) return launch_quantize_group<T, kWide, kNorm, 8, 4>(a, dev, st);
        if (chunks <= 64) return launch_quantize_group<T, kWide, kNorm, 8, 8>(a, dev, st);
        if (chunks <= 128) return launch_quantize_group<T, kWide, kNorm, 8, 16>(a, dev, st);
        if (chunks <= 256) return launch_quantize_group<T, kWide, kNorm, 32, 8>(a, dev, st);
        if (chunks <= 512) return launch_quantize_group<T, kWide, kNorm, 32, 16>(a, dev, st);
        if (chunks <= 1024) return launch_quantize_group<T, kWide, kNorm, 32, 32>(a, dev, st);
        if (chunks <= 2048) return launch_quantize_group<T, kWide, kNorm, 128, 16>(a, dev, st);
        if (chunks <= 4096) return launch_quantize_group<T, kWide, kNorm, 512, 8>(a, dev, st);
    }
    quantize_long_rows_kernel<T, kWide, kNorm><<<grid_of(a.rows, 1, int64_t(dev.num_sms) * 4), 512, 0, st>>>(a);
    return launched();
}

template <typename T>
maxsim_status launch_quantize_any(const QuantizeArgs& a, bool normalize, const HostDevice& dev, cudaStream_t st) {
    constexpr int kVec = Chunk<T, true>::kVec;
    const bool wide = a.cols % kVec == 0 && a.ld_x % kVec == 0 && a.ld_q % kVec == 0 && ptr_aligned(a.x, 16) &&
                      ptr_aligned(a.q, kVec);
    if (normalize) return wide ? launch_quantize<T, true, true>(a, dev, st) : launch_quantize<T, false, true>(a, dev, st);
    return wide ? launch_quantize<T, true, false>(a, dev, st) : launch_quantize<T, false, false>(a, dev, st);
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

// ---------------------------------------------------------------- INT8 linear

constexpr int64_t kPairs = 76;          // CTA pairs of a GB300 (152 SMs): plans do not depend on the device
constexpr uint64_t kTimeoutNs = 2000000000ull;

// Whether the kernels can read rows of K bytes, ld apart, where they are (from
// a 16-byte aligned base): whole 16-byte pieces, and a stride that a TMA
// descriptor can hold.
inline bool rows_direct(int64_t K, int64_t ld) { return K % 16 == 0 && ld % 16 == 0 && ld < (int64_t(1) << 40); }

// linear_few_kernel or the tile kernel. The former takes any product in one
// launch, but reads w once per 32 tokens; a block of it is 16 channels x 32
// tokens. Measured, few / tile, in us: 16 x 16384 x 16384 52 / 55, 8 x 8192 x 8191
// 34 / 45; beyond that by units of a block x 64 of K, and blocks: 32 x 4096 x 4096
// (16,384 units, 256 blocks) 8.3 / 10.1, 128 x 2048 x 2048 (16,384, 512) 8.7 / 10.5,
// 256 x 2048 x 1024 (16,384, 1,024) 9.8 / 8.0, 1024 x 1024 x 512 (16,384, 2,048)
// 12.9 / 7.5, 32 x 16384 x 4096 (65,536, 1,024) 24 / 18. Rows off their 16-byte
// boundaries cost about three times as much: 128 x 1024 x 1023 7.9 / 8.4,
// 3000 x 200 x 301 12.6 / 7.8. The tile kernel's second launch is a further 3 us
// of the caller's time.
constexpr int64_t kFewCost = 20480;
inline bool few_kernel(int64_t M, int64_t N, int64_t K, bool whole) {
    if (M <= 8 || (M <= 16 && whole)) return true;
    const int64_t groups = (M + 31) / 32, tiles = (N + 15) / 16, chunks = (K + 63) / 64;
    if (groups > kFewCost || tiles > kFewCost) return false;
    return groups * tiles * (chunks * (whole ? 1 : 3) + 4) <= kFewCost;
}

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

LinearPlan plan_linear(int64_t M, int64_t N, int64_t K, bool x_direct, bool w_direct) {
    LinearPlan p;
    if (M == 0 || N == 0 || K == 0) return p;
    p.k_pad = (K + 15) / 16 * 16;
    p.few = few_kernel(M, N, K, x_direct && w_direct);
    if (p.few) return p;
    p.swap = N > M;  // the tile kernel's A is the larger operand
    size_t off = 0;
    if (!x_direct && !p.swap) {
        p.off_x = off;
        off = bytes_round_up(off + static_cast<size_t>(M) * p.k_pad, 256);
    }
    if (!w_direct && p.swap) {
        p.off_w = off;
        off = bytes_round_up(off + static_cast<size_t>(N) * p.k_pad, 256);
    }
    const int64_t rows_a = p.swap ? N : M, rows_b = p.swap ? M : N;
    p.off_b = off;
    off = bytes_round_up(off + static_cast<size_t>(rows_b) * p.k_pad * 2, 256);
    // Tile width and slices of K by the time they should take, in cycles:
    // the items of the busiest pair, each its blocks and a start and end,
    // and for slices the kernel that joins them.
    p.kb = static_cast<int32_t>((K + kTileK - 1) / kTileK);
    double best = 0.0;
    for (int tn = 256; tn >= 64; tn /= 2) {
        const int64_t tiles_b = (rows_b + tn - 1) / tn, tiles = (rows_a + kTileM - 1) / kTileM * tiles_b;
        const double block = tn == 256 ? 1050.0 : tn == 128 ? 600.0 : 500.0, ends = tn == 256 ? 3000.0 : 2000.0;
        for (int32_t slices = 1; slices <= std::min(p.kb, 16); ++slices) {
            const int32_t kb_slice = (p.kb + slices - 1) / slices;
            if (slices > 1 && (tiles * slices > 2 * kPairs || (p.kb + kb_slice - 1) / kb_slice != slices)) continue;
            double cost = static_cast<double>((tiles * slices + kPairs - 1) / kPairs) * (kb_slice * block + ends);
            if (slices > 1) cost += 5000.0 + static_cast<double>(M) * N * slices * 4.0 / 1500.0;
            if (best == 0.0 || cost < best) {
                best = cost;
                p.tn = tn;
                p.tiles = tiles;
                p.tiles_b = tiles_b;
                p.slices = slices;
                p.kb_slice = kb_slice;
            }
        }
    }
    // a single tile of B for several tiles of A on every pair
    p.keep_b = !p.swap && p.slices == 1 && p.tiles_b == 1 && p.tiles > kPairs &&
               ((p.tn == 128 && p.kb <= TileCfg<128, true>::kStagesB) || (p.tn == 64 && p.kb <= TileCfg<64, true>::kStagesB));
    if (p.slices > 1) {
        p.off_partial = off;
        off = bytes_round_up(off + static_cast<size_t>(p.slices) * M * N * 4, 256);
    }
    p.bytes = off;
    return p;
}

// Rows of K elements, ld bytes apart, in boxes of 128 bytes x box_rows with the 128-byte swizzle.
bool encode_k_rows(EncodeTiledFn encode, CUtensorMap* map, CUtensorMapDataType type, int elem, const void* base,
                   int64_t K, int64_t rows, int64_t ld, uint32_t box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
    const cuuint32_t box[2] = {128u / static_cast<cuuint32_t>(elem), box_rows}, estr[2] = {1, 1};
    return encode(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

template <typename T, int kTN, bool kSwap, bool kKeepB>
maxsim_status launch_tile(const LinearPlan& p, const LinearArgs& l, const __half* b16, bool a_prepared, int32_t* partial,
                          const HostDevice& dev, cudaStream_t st) {
    auto kern = linear_tile_kernel<T, kTN, kSwap, kKeepB>;
    constexpr size_t kSmem = tile_smem_bytes<kTN, kKeepB>();
    static_assert(kSmem <= 232448, "shared memory of one SM");
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
    a.vec_out = p.slices > 1 ? l.N % 4 == 0
                             : ptr_aligned(l.out, 16) && l.ld_out * static_cast<int64_t>(sizeof(T)) % 16 == 0;
    a.a_prepared = a_prepared;
    a.status = dev.status;
    a.timeout_ns = kTimeoutNs;
    CUtensorMap ta, tb;
    if (!encode_k_rows(dev.encode, &ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kSwap ? l.w : l.x, l.K, a.rows_a,
                       kSwap ? l.ld_w : l.ld_x, 128) ||
        !encode_k_rows(dev.encode, &tb, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, b16, p.k_pad, a.rows_b, p.k_pad * 2,
                       TileCfg<kTN, kKeepB>::kBRows))
        return MAXSIM_ERR_CUDA;
    return launch_after(kern, static_cast<unsigned>(2 * std::min<int64_t>(a.items, std::max(1, dev.num_sms / 2))), kTileThreads,
                        kSmem, 2, st, ta, tb, a);
}

template <typename T, bool kSwap>
maxsim_status launch_tile_width(const LinearPlan& p, const LinearArgs& l, const __half* b16, bool a_prepared, int32_t* partial,
                                const HostDevice& dev, cudaStream_t st) {
    if constexpr (!kSwap) {
        if (p.keep_b && p.tn == 128) return launch_tile<T, 128, false, true>(p, l, b16, a_prepared, partial, dev, st);
        if (p.keep_b) return launch_tile<T, 64, false, true>(p, l, b16, a_prepared, partial, dev, st);
    }
    if (p.tn == 256) return launch_tile<T, 256, kSwap, false>(p, l, b16, a_prepared, partial, dev, st);
    if (p.tn == 128) return launch_tile<T, 128, kSwap, false>(p, l, b16, a_prepared, partial, dev, st);
    return launch_tile<T, 64, kSwap, false>(p, l, b16, a_prepared, partial, dev, st);
}

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
    rc = p.swap ? launch_tile_width<T, true>(p, l, b16, prepared, partial, dev, st)
                : launch_tile_width<T, false>(p, l, b16, prepared, partial, dev, st);
    if (rc != MAXSIM_OK || p.slices == 1) return rc;
    return launch_after(linear_join_kernel<T>, join_grid, 256, 0, 1, st, l, const_cast<const int32_t*>(partial), p.slices);
}

}  // namespace

size_t linear_int8_ws_bytes(int64_t M, int64_t N, int64_t K, int64_t ld_x, int64_t ld_w) {
    if (M < 0 || N < 0 || K < 0 || ld_x < 0 || ld_w < 0 || M > kLinearMaxRows || N > kLinearMaxRows || K > kLinearMaxK)
        return static_cast<size_t>(-1);
    return plan_linear(M, N, K, rows_direct(K, ld_x), rows_direct(K, ld_w)).bytes;
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
    const QuantizeArgs a{x, q, scale, rows, ld_x, ld_q, static_cast<int32_t>(cols)};
    if (dtype == MAXSIM_F16) return launch_quantize_any<__half>(a, normalize != 0, dev, st);
    if (dtype == MAXSIM_BF16) return launch_quantize_any<__nv_bfloat16>(a, normalize != 0, dev, st);
    return launch_quantize_any<float>(a, normalize != 0, dev, st);
}

maxsim_status maxsim_linear_int8(const int8_t* x, int64_t ld_x, const float* x_scale, const int8_t* w, int64_t ld_w,
                                 const float* w_scale, const float* bias, int64_t M, int64_t N, int64_t K,
                                 maxsim_dtype out_dtype, void* out, int64_t ld_out, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    if (!any_dtype(out_dtype) || M < 0 || N < 0 || K < 0) return MAXSIM_ERR_INVALID_ARG;
    if (!rows_fit(M, K, ld_x) || !rows_fit(N, K, ld_w) || !rows_fit(M, N, ld_out)) return MAXSIM_ERR_INVALID_ARG;
    if (M > kLinearMaxRows || N > kLinearMaxRows || K > kLinearMaxK) return MAXSIM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return MAXSIM_OK;
    if (!out || !ptr_aligned(out, elem_bytes(out_dtype))) return MAXSIM_ERR_INVALID_ARG;
    if (!x_scale || !w_scale || !ptr_aligned(x_scale, 4) || !ptr_aligned(w_scale, 4) || !ptr_aligned(bias, 4))
        return MAXSIM_ERR_INVALID_ARG;
    if (K > 0 && (!x || !w)) return MAXSIM_ERR_INVALID_ARG;
    const bool x_direct = rows_direct(K, ld_x) && ptr_aligned(x, 16), w_direct = rows_direct(K, ld_w) && ptr_aligned(w, 16);
    const LinearPlan p = plan_linear(M, N, K, x_direct, w_direct);
    if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes || !ptr_aligned(workspace, 256)))
        return MAXSIM_ERR_WORKSPACE;
    HostDevice dev;
    const maxsim_status rc = host_device(&dev);
    if (rc != MAXSIM_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t* ws8 = static_cast<uint8_t*>(workspace);
    const LinearArgs l{x, w, ld_x, ld_w, ld_out, x_scale, w_scale, bias, out,
                       static_cast<int32_t>(M), static_cast<int32_t>(N), static_cast<int32_t>(K)};
    if (out_dtype == MAXSIM_F16) return run_linear<__half>(p, l, x_direct, w_direct, ws8, dev, st);
    if (out_dtype == MAXSIM_BF16) return run_linear<__nv_bfloat16>(p, l, x_direct, w_direct, ws8, dev, st);
    return run_linear<float>(p, l, x_direct, w_direct, ws8, dev, st);
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
