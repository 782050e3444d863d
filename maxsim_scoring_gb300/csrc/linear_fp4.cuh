// out[m, n] = (sum_k x[m, k] w[n, k]) * x_scale[m] * w_scale[n] + bias[n] for
// rows of 4-bit floating-point values with block scales (fp4_kernels.cuh).
//
// The codes and their block scales go to the tensor cores as they are:
// tcgen05.mma.kind::mxf4nvf4 multiplies blocks of 16 (E4M3 scales) or 32 (E8M0)
// codes with their scales and sums in fp32.
#pragma once

#include <cstdint>
#include <type_traits>

#include "fp4_kernels.cuh"
#include "ptx.cuh"
#include "tile_store.cuh"

namespace maxsim {

struct LinearFp4Args {
    const uint8_t* x;
    const uint8_t* w;
    const uint8_t* x_block;
    const uint8_t* w_block;
    int64_t ld_x, ld_w, ld_out;  // bytes, bytes, elements
    const float* x_scale;        // NULL: 1
    const float* w_scale;        // NULL: 1
    const float* bias;           // NULL: none
    void* out;
    int32_t M, N, K;             // K a multiple of 32
    int32_t words;               // scale words of a row
};

constexpr int kFp4TileM = 256;      // rows of A per tile: 128 on each CTA of a pair
constexpr int kFp4TileK = 256;      // values of K per stage: 128 bytes of a row
constexpr int kFp4Threads = 384;    // warp 0 TMA, warp 1 MMA (odd CTA: reports what landed), warps 4-11 epilogue
constexpr int kFp4EpiWarp0 = 4;
constexpr int kFp4MaxSplits = 4;

template <int kTN>
struct Fp4Cfg {
    static constexpr int kA = 128 * 128;                     // this CTA's 128 rows of A
    static constexpr int kBRows = kTN / 2;                   // rows of B per CTA
    static constexpr int kB = kBRows * 128;
    static constexpr int kBTiles = kTN > 128 ? kTN / 128 : 1;  // scale tiles (128 rows) of a tile's rows of B
    static constexpr int kSfa = 4 * 512, kSfb = kBTiles * 4 * 512;  // at most: block 16
    static constexpr int kStage = kA + kB + kSfa + kSfb;
    static constexpr int kStages = kTN == 256 ? 5 : kTN == 128 ? 6 : 8;
    static constexpr int kAcc = kTN == 256 ? 1 : 2;          // accumulator buffers
    static constexpr int kSfCols = 4 * 4 + 4 * 4 * kBTiles;  // columns of tensor memory for a stage's scales
    static_assert(kAcc * kTN + kStages * kSfCols <= 512, "tensor memory");
};

struct LinearFp4TileArgs {
    LinearFp4Args l;
    int64_t items;      // tiles
    int32_t rows_a;     // rows of A (tokens, or channels when swapped)
    int32_t rows_b;
    int32_t tiles_b;
    int32_t kb;         // stages of K
    int32_t kb_part;    // f32 outputs: stages summed in one accumulator
    int32_t splits;     // pairs of a cluster that share a tile's K
    int32_t kb_split;   // stages of each
    int32_t block;      // 16 or 32
    int* status;
    uint64_t timeout_ns;
};

struct alignas(16) Fp4Ctl {
    uint64_t full[8], empty[8];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    volatile int32_t abort;
};

template <int kTN>
constexpr size_t fp4_smem_bytes() {
    using C = Fp4Cfg<kTN>;
    return 1024 + static_cast<size_t>(C::kStages) * C::kStage + 8 * 4096 + sizeof(Fp4Ctl);
}

// 3-D tiled load (x innermost).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Shared-memory descriptor of a tile of scale words: 32 rows of 16 bytes, no
// swizzle, eight rows (128 bytes) a core matrix.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(128 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    return d;
}

// Copies a tile of scale words (512 bytes) to four columns of tensor memory, in
// all four lane quarters, on both CTAs of the pair from their own shared memory;
// from the elected lane.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t sdesc) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(sdesc)
        : "memory");
}

// Instruction descriptor of kind::mxf4nvf4: [4,6) B's scale word byte, [7,10)
// and [10,12) A's and B's type (1 = E2M1), [17,23) N >> 3, [23] scales E8M0
// instead of E4M3, [24,29) M >> 4, [29,31) A's scale word byte. Both operands K-major.
__host__ __device__ constexpr uint32_t idesc_fp4(uint32_t M, uint32_t N, bool e8m0, uint32_t byte) {
    return (byte << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | (e8m0 ? 1u << 23 : 0u) | ((M >> 4) << 24) | (byte << 29);
}

// The four K = 64 steps of a stage, from the elected lane: 32 bytes of A's and
// B's rows a step (K-major, 128-byte swizzle). With blocks of 16 a step takes a
// scale word of each row, with blocks of 32 half a word.
template <uint32_t kSfbStep>
__device__ __forceinline__ void mma_stage16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p0, pt;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t.reg .b32 s1, s2, s3, t1, t2, t3;\n\t"
        "setp.ne.b32 p0, %6, 0;\n\tsetp.eq.b32 pt, %6, %6;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "add.u32 s1, %4, 4;\n\tadd.u32 s2, %4, 8;\n\tadd.u32 s3, %4, 12;\n\t"
        "add.u32 t1, %5, %7;\n\tadd.u32 t2, %5, %8;\n\tadd.u32 t3, %5, %9;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], a1, b1, %3, [s1], [t1], pt;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], a2, b2, %3, [s2], [t2], pt;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], a3, b3, %3, [s3], [t3], pt;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kSfbStep), "n"(2 * kSfbStep), "n"(3 * kSfbStep)
        : "memory");
}
template <uint32_t kSfbStep>
__device__ __forceinline__ void mma_stage32(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t idesc_hi, uint32_t sfa, uint32_t sfb,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p0, pt;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t.reg .b32 s1, t1;\n\t"
        "setp.ne.b32 p0, %7, 0;\n\tsetp.eq.b32 pt, %7, %7;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "add.u32 s1, %5, 4;\n\tadd.u32 t1, %6, %8;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], a1, b1, %4, [%5], [%6], pt;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], a2, b2, %3, [s1], [t1], pt;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], a3, b3, %4, [s1], [t1], pt;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(idesc_hi), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kSfbStep)
        : "memory");
}

// Every thread of every CTA of the cluster, whatever its warp's other threads do.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// One tile is 256 rows of A (128 on each CTA of a pair) x kTN rows of B (half on
// each). A is the larger operand: x, or w when kSwap.
//  * warp 0 brings stages of 256 values of K by TMA: its CTA's rows of A and B
//    (128-byte swizzle) with the scale tiles of its rows of A and of all the
//    tile's rows of B, which both CTAs' MMA halves need. What lies outside the
//    operands reads as code 0 with scale 0;
//  * warp 1 of the even CTA copies a stage's scales to tensor memory and issues
//    its MMAs (M = 256, N = kTN, K = 64), which the hardware keeps in this order;
//    warp 1 of the odd CTA reports to it what landed there;
//  * eight epilogue warps scale, add the bias, round once and store, as those of
//    linear_tile_kernel do.
// kRows16: rows of out start on 16-byte boundaries, and 16-bit ones end there.
// splits > 1 (few tiles): the pairs of a cluster share a tile's K; the others'
// sums pass to the first pair's shared memory and are added in their order.
template <typename T, int kTN, bool kSwap, bool kRows16>
__global__ void __launch_bounds__(kFp4Threads, 1)
linear_fp4_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_sfa,
                  const __grid_constant__ CUtensorMap tm_sfb, const __grid_constant__ CUtensorMap tm_out, const LinearFp4TileArgs a) {
    using C = Fp4Cfg<kTN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* s_a = smem;
    uint8_t* s_b = s_a + C::kStages * C::kA;
    uint8_t* s_sfa = s_b + C::kStages * C::kB;
    uint8_t* s_sfb = s_sfa + C::kStages * C::kSfa;
    uint8_t* s_out = s_sfb + C::kStages * C::kSfb;
    Fp4Ctl* ctl = reinterpret_cast<Fp4Ctl*>(s_out + 8 * 4096);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank(), rank = crank & 1u, even = crank & ~1u;
    const int32_t split = static_cast<int32_t>(crank >> 1);
    const int32_t words = a.block == 16 ? 4 : 2;  // scale words of a stage
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), rank == 0 ? 2 : 1);  // its own TMA; even CTA: and the odd CTA's report
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&ctl->acc_full[b]), 1);
            mbar_init(smem_u32(&ctl->acc_empty[b]), 16);  // eight warps of each CTA
        }
        mbar_init(smem_u32(&ctl->mma_done), 1);
        ctl->abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
        tma_prefetch_desc(&tm_sfa);
        tma_prefetch_desc(&tm_sfb);
    }
    if (warp == 1) {
        tmem_alloc<2>(smem_u32(&ctl->tmem_base), 512);
        tmem_relinquish<2>();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // barriers of all CTAs exist before any remote arrival
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    const uint32_t ctas = 2u * static_cast<uint32_t>(a.splits);
    const int64_t first = blockIdx.x / ctas, step = gridDim.x / ctas;
    const int32_t kb0 = split * a.kb_split, kb1 = min(a.kb, kb0 + a.kb_split);

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA
        if (lane == 0) {
            const uint32_t bytes = static_cast<uint32_t>(C::kA + C::kB) + static_cast<uint32_t>(words) * 512u * (1 + C::kBTiles);
            int32_t stage = 0;
            uint32_t phase = 0;
            int64_t issued = 0;
            bool ok = true;
            for (int64_t it = first; it < a.items && ok; it += step) {
                const int64_t row = it / a.tiles_b;
                const int32_t a0 = static_cast<int32_t>(row * kFp4TileM) + static_cast<int32_t>(rank) * 128;
                const int32_t b0 = static_cast<int32_t>(it - row * a.tiles_b) * kTN;
                for (int32_t kb = kb0; kb < kb1; ++kb) {
                    if (!tile_wait(a, ctl, &ctl->empty[stage], phase ^ 1u)) { ok = false; break; }
                    const uint32_t bar = smem_u32(&ctl->full[stage]);
                    mbar_arrive_expect_tx(bar, bytes);
                    tma_load_2d(smem_u32(s_a + stage * C::kA), &tm_a, bar, kb * 128, a0);
                    tma_load_2d(smem_u32(s_b + stage * C::kB), &tm_b, bar, kb * 128, b0 + static_cast<int32_t>(rank) * C::kBRows);
                    tma_load_3d(smem_u32(s_sfa + stage * C::kSfa), &tm_sfa, bar, 0, kb * words, a0 >> 7);
                    tma_load_3d(smem_u32(s_sfb + stage * C::kSfb), &tm_sfb, bar, 0, kb * words, b0 >> 7);
                    ++issued;
                    if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                }
            }
            if (ctl->abort) {  // the copies still in flight land before the CTA leaves
                const int64_t n = issued < C::kStages ? issued : C::kStages;
                for (int64_t i = 0; i < n; ++i) {
                    if (--stage < 0) { stage = C::kStages - 1; phase ^= 1u; }
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait(smem_u32(&ctl->full[stage]), phase) && global_timer_ns() - t0 < a.timeout_ns) {}
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        int32_t stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        if (rank == 0) {
            // ------------------------------------------------------------ MMA (even CTA)
            const uint64_t a_desc = sdesc_k_sw128(smem_u32(s_a)), b_desc = sdesc_k_sw128(smem_u32(s_b));
            const uint64_t fa_desc = sdesc_scales(smem_u32(s_sfa)), fb_desc = sdesc_scales(smem_u32(s_sfb));
            const uint32_t sf0 = tmem + C::kAcc * kTN;
            const uint16_t both = static_cast<uint16_t>(3u << even);
            const bool b16 = a.block == 16;
            const uint32_t idesc = idesc_fp4(kFp4TileM, kTN, !b16, 0), idesc_hi = idesc_fp4(kFp4TileM, kTN, !b16, 2);
            int32_t buf = 0;
            uint32_t buf_phase = 0;
            for (int64_t it = first; it < a.items && ok; it += step) {
                // kTN = 64: the odd tiles' rows are the upper half of a scale tile
                const uint32_t sfb_off = kTN == 64 ? static_cast<uint32_t>((it % a.tiles_b) & 1) * 2u : 0u;
                int32_t s0 = kb0;
                do {  // a run of stages that are summed in one accumulator
                    const int32_t s1 = std::is_same_v<T, float> ? min(kb1, s0 + a.kb_part) : kb1;
                    if (!tile_wait_warp<true>(a, ctl, &ctl->acc_empty[buf], buf_phase ^ 1u)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t d = tmem + static_cast<uint32_t>(buf * kTN);
                    for (int32_t kb = s0; kb < s1; ++kb) {
                        if (!tile_wait_warp<true>(a, ctl, &ctl->full[stage], phase)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t sfa = sf0 + static_cast<uint32_t>(stage * C::kSfCols), sfb = sfa + 16;
                        const uint64_t fa = fa_desc + static_cast<uint64_t>((stage * C::kSfa) >> 4);
                        const uint64_t fb = fb_desc + static_cast<uint64_t>((stage * C::kSfb) >> 4);
                        const uint64_t da = a_desc + static_cast<uint64_t>((stage * C::kA) >> 4);
                        const uint64_t db = b_desc + static_cast<uint64_t>((stage * C::kB) >> 4);
                        for (int32_t j = 0; j < words; ++j) {
                            copy_scales(sfa + 4 * j, fa + 32 * j);
#pragma unroll
                            for (int r = 0; r < C::kBTiles; ++r)
                                copy_scales(sfb + (j * C::kBTiles + r) * 4, fb + 32 * (r * words + j));
                        }
                        if (b16) mma_stage16<4 * C::kBTiles>(d, da, db, idesc, sfa, sfb + sfb_off, kb > s0 ? 1u : 0u);
                        else mma_stage32<4 * C::kBTiles>(d, da, db, idesc, idesc_hi, sfa, sfb + sfb_off, kb > s0 ? 1u : 0u);
                        mma_commit_elect<2>(smem_u32(&ctl->empty[stage]), both);
                        if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                    }
                    if (!ok) break;
                    mma_commit_elect<2>(smem_u32(&ctl->acc_full[buf]), both);
                    if (++buf == C::kAcc) { buf = 0; buf_phase ^= 1u; }
                    s0 = s1;
                } while (std::is_same_v<T, float> && s0 < kb1);
            }
            // every MMA issued above completes before the CTA leaves
            mma_commit_elect<2>(smem_u32(&ctl->mma_done), static_cast<uint16_t>(1u << even));
            if (lane == 0) {
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(smem_u32(&ctl->mma_done), 0) && global_timer_ns() - t0 < a.timeout_ns) {}
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------ odd CTA: reports what landed
            for (int64_t it = first; it < a.items && ok; it += step) {
                for (int32_t kb = kb0; kb < kb1; ++kb) {
                    if (!tile_wait_warp(a, ctl, &ctl->full[stage], phase)) { ok = false; break; }
                    if (lane == 0) mbar_arrive_remote(map_shared_rank(smem_u32(&ctl->full[stage]), even));
                    if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                }
            }
        }
    } else if (warp >= kFp4EpiWarp0) {
        // ---------------------------------------------------------------- epilogue
        // A warp owns 32 rows of A (a lane each) and half of the tile's columns.
        const int q = warp & 3, half = (warp - kFp4EpiWarp0) >> 2;
        constexpr int kCols = kTN / 2, kChunks = kCols / 32;
        constexpr bool kHold = sizeof(T) == 2, kTma = kHold && kRows16 && !kSwap;
        uint8_t* stage = s_out + (warp - kFp4EpiWarp0) * 4096;
        float* tab = reinterpret_cast<float*>(stage);  // scales of the kCols columns, then biases
        const int64_t ld = a.l.ld_out;
        const float* scale_a = kSwap ? a.l.w_scale : a.l.x_scale;
        const float* scale_b = kSwap ? a.l.x_scale : a.l.w_scale;
        T* out = static_cast<T*>(a.l.out);
        int32_t buf = 0;
        uint32_t buf_phase = 0;
        for (int64_t it = first; it < a.items; it += step) {
            const int64_t row = it / a.tiles_b;
            const int64_t ra0 = row * kFp4TileM + rank * 128 + q * 32, rb0 = (it - row * a.tiles_b) * kTN + half * kCols;
            const int row_n = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(32), a.rows_a - ra0)));
            const bool in_a = lane < row_n;
            const float sa = scale_a && in_a ? __ldg(scale_a + ra0 + lane) : 1.f;
            const float bias_a = kSwap && a.l.bias && in_a ? __ldg(a.l.bias + ra0 + lane) : 0.f;
            float sb[kChunks], bias[kChunks];
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int64_t i = rb0 + c * 32 + lane;
                sb[c] = scale_b && i < a.rows_b ? __ldg(scale_b + i) : 1.f;
                bias[c] = !kSwap && a.l.bias && i < a.rows_b ? __ldg(a.l.bias + i) : 0.f;
            }
            if constexpr (kTma) {  // the table is written where the last tile's stores read
                if (lane == 0) bulk_wait_read();
                __syncwarp();
            }
            if constexpr (kHold) {
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    tab[c * 32 + lane] = sb[c];
                    if constexpr (!kSwap) tab[kCols + c * 32 + lane] = bias[c];
                }
                __syncwarp();
            }
            const float2 sa2 = make_float2(sa, sa);
            const uint32_t src0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * kCols);
            float sum[kHold ? 1 : kCols];
            uint32_t held[kHold ? kChunks : 1][16];
            // other pairs' sums: [splits - 1][kTN][128], of this lane's row and first column
            const float* parts = reinterpret_cast<const float*>(s_a) + (half * kCols) * 128 + q * 32 + lane;
            if (a.splits > 1) {
                const bool done = tile_wait_warp(a, ctl, &ctl->acc_full[buf], buf_phase);
                tc_fence_after();
                cluster_arrive();  // all MMAs of the cluster are done: the first pair's stages are free
                cluster_wait();
                if (split > 0 && done) {
                    const uint32_t to = map_shared_rank(smem_u32(parts), rank) + static_cast<uint32_t>(split - 1) * (kTN * 128 * 4);
                    for (int c = 0; c < kCols; c += 16) {
                        float v[16];
                        tmem_ld16(src0 + c, v);
                        tmem_wait_ld16(v);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + static_cast<uint32_t>(c + i) * 512u), "f"(v[i]) : "memory");
                    }
                }
                cluster_arrive();
                cluster_wait();
                if (split > 0 || !done) break;
            }
            bool ok = true;
            int32_t s0 = kb0;
            do {  // runs of stages, as the MMAs
                if (a.splits == 1) {
                    if (!(ok = tile_wait_warp(a, ctl, &ctl->acc_full[buf], buf_phase))) break;
                    tc_fence_after();
                }
                const uint32_t src = src0 + static_cast<uint32_t>(buf * kTN);
                // one part is in flight while another is worked on
                constexpr int kLoads = kCols / 16;
                float v[2][16];
                tmem_ld16(src, v[0]);
#pragma unroll
                for (int c = 0; c < kLoads; ++c) {
                    tmem_wait_ld16(v[c & 1]);
                    if (c + 1 < kLoads) {
                        tmem_ld16(src + (c + 1) * 16, v[(c + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(map_shared_rank(smem_u32(&ctl->acc_empty[buf]), even));
                    }
                    float (&u)[16] = v[c & 1];
                    if (a.splits > 1) {
                        for (int32_t s = 0; s + 1 < a.splits; ++s)
#pragma unroll
                            for (int i = 0; i < 16; ++i) u[i] += parts[s * (kTN * 128) + (c * 16 + i) * 128];
                    }
                    if constexpr (kHold) {
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const float4 s4 = *reinterpret_cast<const float4*>(tab + c * 16 + i);
                            const float4 b4 = kSwap ? make_float4(bias_a, bias_a, bias_a, bias_a)
                                                    : *reinterpret_cast<const float4*>(tab + kCols + c * 16 + i);
                            const float2 lo = fma2(mul2(make_float2(u[i], u[i + 1]), sa2), make_float2(s4.x, s4.y), make_float2(b4.x, b4.y));
                            const float2 hi = fma2(mul2(make_float2(u[i + 2], u[i + 3]), sa2), make_float2(s4.z, s4.w), make_float2(b4.z, b4.w));
                            held[c / 2][(c & 1) * 8 + i / 2] = pack2<T>(lo.x, lo.y);
                            held[c / 2][(c & 1) * 8 + i / 2 + 1] = pack2<T>(hi.x, hi.y);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[c * 16 + i] = s0 == kb0 ? u[i] : sum[c * 16 + i] + u[i];
                    }
                }
                if (++buf == C::kAcc) { buf = 0; buf_phase ^= 1u; }
                s0 += a.kb_part;
            } while (!kHold && s0 < kb1);
            if (!ok) break;
            if constexpr (kHold) {
                store_held<T, kCols, kSwap, kTma>(held, stage, out, ld, ra0, rb0, a.rows_b, row_n, &tm_out);
            } else {
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const int64_t rb = rb0 + c * 32;
                    if (row_n == 0 || rb >= a.rows_b) break;
                    const float* v = sum + c * 32;
                    if constexpr (kSwap) {
                        const int n = static_cast<int>(min(static_cast<int64_t>(32), a.rows_b - rb));
                        float* p = out + rb * ld + ra0 + lane;
#pragma unroll
                        for (int i = 0; i < 32; ++i, p += ld) {
                            const float y = __fmaf_rn(v[i] * __shfl_sync(0xffffffffu, sb[c], i), sa, bias_a);
                            if (i < n && in_a) *p = y;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<float4*>(stage + staged(lane, i)) =
                                make_float4(v[4 * i] * sa, v[4 * i + 1] * sa, v[4 * i + 2] * sa, v[4 * i + 3] * sa);
                        __syncwarp();
                        if constexpr (kRows16) {
                            float ws[4], bs[4];  // this lane's four channels
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                ws[j] = __shfl_sync(0xffffffffu, sb[c], 4 * (lane & 7) + j);
                                bs[j] = __shfl_sync(0xffffffffu, bias[c], 4 * (lane & 7) + j);
                            }
                            const int64_t n0 = rb + 4 * (lane & 7);
                            const int n = static_cast<int>(min(static_cast<int64_t>(4), a.rows_b - n0));
                            int64_t at = (ra0 + (lane >> 3)) * ld + n0;
#pragma unroll
                            for (int i = 0; i < 8; ++i, at += 4 * ld) {
                                const float4 y = *reinterpret_cast<const float4*>(stage + staged(4 * i + (lane >> 3), lane & 7));
                                if (4 * i + (lane >> 3) < row_n)
                                    store4(out + at, n, __fmaf_rn(y.x, ws[0], bs[0]), __fmaf_rn(y.y, ws[1], bs[1]),
                                           __fmaf_rn(y.z, ws[2], bs[2]), __fmaf_rn(y.w, ws[3], bs[3]));
                            }
                        } else {  // rows off their 16-byte boundaries: a row at a time, a lane per column
                            const bool in_b = rb + lane < a.rows_b;
                            const uint8_t* from = stage + (lane & 3) * 4;
                            int64_t at = ra0 * ld + rb + lane;
#pragma unroll 8
                            for (int r = 0; r < row_n; ++r, at += ld) {
                                const float y = *reinterpret_cast<const float*>(from + staged(r, lane >> 2));
                                if (in_b) out[at] = __fmaf_rn(y, sb[c], bias[c]);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
        }
        if (kTma && lane == 0) bulk_wait();
    }
    if (a.splits > 1 && warp < kFp4EpiWarp0) {  // the epilogue warps' two meetings
        cluster_arrive();
        cluster_wait();
        cluster_arrive();
        cluster_wait();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // no CTA leaves while another may still touch it
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc<2>(tmem, 512);
    }
}

// K = 0: the bias.
template <typename T>
__global__ void __launch_bounds__(256) linear_fp4_bias_kernel(const LinearFp4Args l) {
    const int64_t n_out = static_cast<int64_t>(l.M) * l.N;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n_out; i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t m = i / l.N, n = i - m * l.N;
        // a NaN row scale counts here too
        const float v = 0.f * (l.x_scale ? l.x_scale[m] : 1.f) * (l.w_scale ? l.w_scale[n] : 1.f);
        static_cast<T*>(l.out)[m * l.ld_out + n] = from_f32<T>(l.bias ? v + l.bias[n] : v);
    }
}

}  // namespace maxsim
