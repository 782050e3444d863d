// Host side of the INT8 linear (include/maxsim.h): argument validation and the
// plan; the launches are linear_launch.cuh's.
#include <algorithm>
#include <cstdint>

#include "linear_launch.cuh"

namespace maxsim {

extern template maxsim_status run_linear<__half>(const LinearPlan&, LinearArgs, bool, bool, uint8_t*, const HostDevice&, cudaStream_t);
extern template maxsim_status run_linear<__nv_bfloat16>(const LinearPlan&, LinearArgs, bool, bool, uint8_t*, const HostDevice&, cudaStream_t);
extern template maxsim_status run_linear<float>(const LinearPlan&, LinearArgs, bool, bool, uint8_t*, const HostDevice&, cudaStream_t);

namespace {

constexpr int64_t kLinearMaxK = 131071;             // 131071 * 128 * 128 < 2^31
constexpr int64_t kLinearMaxRows = kI32Max - 1023;  // a tile past the last row still has 32-bit coordinates
constexpr int64_t kPairs = 76;          // CTA pairs of a GB300 (152 SMs): plans do not depend on the device

// Whether the kernels can read rows of K bytes, ld apart, where they are (from
// a 16-byte aligned base): whole 16-byte pieces, and a stride that a TMA
// descriptor can hold.
inline bool rows_direct(int64_t K, int64_t ld) { return K % 16 == 0 && ld % 16 == 0 && ld < (int64_t(1) << 40); }

// linear_few_kernel or the tile kernel. The former takes any product in one
// launch, but reads w once per 32 tokens; a block of it is 16 channels x 32
// tokens. Up to 16 tokens it wins (few / tile, us on the GPU): 16 x 16384 x
// 16384 52 / 55, 8 x 8192 x 8191 34 / 45. Beyond, by the cost below (blocks x
// chunks of K, three times as much for rows off their 16-byte boundaries):
//                       cost   GPU          call, one after another
//   128 x 1024 x 1024    5120   4.5 /  7.7   12 / 22
//   512 x 512 x 1024    10240   6.1 /  8.0   13 / 21
//   900 x 900 x 256     13224  10.0 /  6.5   12 / 21
//   2048 x 512 x 256    16384  12.0 /  6.0   14 / 22
//   32 x 4096 x 4096    17408   8.2 /  9.7   12 / 24
//   256 x 2048 x 1024   20480   9.5 /  7.8   13 / 22
//   1024 x 1024 x 512   24576  12.7 /  6.8   15 / 21
//   64 x 1000 x 4095    24696  11.8 /  9.7   14 / 24
// The tile kernel's second launch and workspace are 7 to 9 us of an eager call,
// so up to the limit a call is shorter through the few kernel even where its
// GPU time, all that counts in a CUDA graph or a full queue, is up to 6 us
// longer (many tokens, short K).
constexpr int64_t kFewCost = 20480;
inline bool few_kernel(int64_t M, int64_t N, int64_t K, bool whole) {
    if (M <= 8 || (M <= 16 && whole)) return true;
    const int64_t groups = (M + 31) / 32, tiles = (N + 15) / 16, chunks = (K + 63) / 64;
    if (groups > kFewCost || tiles > kFewCost) return false;
    return groups * tiles * (chunks * (whole ? 1 : 3) + 4) <= kFewCost;
}

LinearPlan plan_linear(int64_t M, int64_t N, int64_t K, bool x_direct, bool w_direct, bool out32) {
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
            // no parts in 256 columns; slices of few blocks, which could do without, are never the cheapest there
            if (tn == 256 && (slices > 1 || (out32 && parts_needed(kb_slice)))) continue;
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

}  // namespace

size_t linear_int8_ws_bytes(int64_t M, int64_t N, int64_t K, int64_t ld_x, int64_t ld_w) {
    if (M < 0 || N < 0 || K < 0 || ld_x < 0 || ld_w < 0 || M > kLinearMaxRows || N > kLinearMaxRows || K > kLinearMaxK)
        return static_cast<size_t>(-1);
    const bool x_direct = rows_direct(K, ld_x), w_direct = rows_direct(K, ld_w);
    return std::max(plan_linear(M, N, K, x_direct, w_direct, false).bytes, plan_linear(M, N, K, x_direct, w_direct, true).bytes);
}

}  // namespace maxsim

using namespace maxsim;

extern "C" {

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
    const LinearPlan p = plan_linear(M, N, K, x_direct, w_direct, out_dtype == MAXSIM_F32);
    if (p.tiles * p.slices > kI32Max) return MAXSIM_ERR_UNSUPPORTED;
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

}  // extern "C"
