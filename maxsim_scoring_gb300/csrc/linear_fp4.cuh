// out[m, n] = (sum_k x[m, k] w[n, k]) * (x_scale[m] * w_scale[n]) + bias[n] for
// rows of 4-bit floating-point values with block scales (fp4_kernels.cuh).
//
// The codes and their block scales go to the tensor cores as they are:
// tcgen05.mma.kind::mxf4nvf4 multiplies blocks of 16 (E4M3 scales) or 32 (E8M0)
// codes with their scales and sums in fp32.
#pragma once

#include <cstdint>
#include <type_traits>

#include "fp4_kernels.cuh"
#include "linear_fp4_plan.h"
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

constexpr int kFp4Threads = 384;    // warps 0 and 3 TMA, warps 1 and 2 MMA and scales (even CTA), warps 4-11 epilogue
constexpr int kFp4EpiWarp0 = 4;
// Registers a thread: the launch gives kFp4Regs, of which the first warpgroup
// hands some to the epilogue's two, which hold a tile's sums between the
// accumulator's hand-over and the stores.
constexpr int kFp4Regs = 168, kFp4RegsCtl = 80, kFp4RegsEpi = 208;
static_assert(kFp4RegsCtl + 2 * kFp4RegsEpi <= 3 * kFp4Regs, "register split");

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
    int32_t splits;     // pairs of a cluster that share a tile's K
    int32_t kb_split;   // stages of each
    int32_t block;      // 16 or 32
    int prefetch;       // tiles of A ahead
    int* status;
    uint64_t timeout_ns;
};

struct alignas(16) Fp4Ctl {
    uint64_t full[8], empty[8], scales[8];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t mma_done, copies_done;
    uint32_t tmem_base;
    volatile int32_t abort;
};

template <int kTN>
constexpr size_t fp4_smem_bytes() {
    using C = Fp4Cfg<kTN>;
    return 1024 + static_cast<size_t>(C::kStages) * C::kStage + 8 * 4096 + sizeof(Fp4Ctl);
}

// Tiled loads into this CTA's shared memory whose bytes count on a barrier of
// either CTA of the pair (its shared::cluster address); x innermost.
__device__ __forceinline__ void tma_load_pair_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_pair_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Tiled prefetches into L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int32_t x, int32_t y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int32_t x, int32_t y, int32_t z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z)
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

// Instruction descriptor of kind::mxf4nvf4: [4,6) B's scale word byte, [7,10)
// and [10,12) A's and B's type (1 = E2M1), [17,23) N >> 3, [23] scales E8M0
// instead of E4M3, [24,29) M >> 4, [29,31) A's scale word byte. Both operands K-major.
__host__ __device__ constexpr uint32_t idesc_fp4(uint32_t M, uint32_t N, bool e8m0, uint32_t byte) {
    return (byte << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | (e8m0 ? 1u << 23 : 0u) | ((M >> 4) << 24) | (byte << 29);
}

// The copies and the MMAs of a stage, from the elected lane, in one asm block
// each (issued one by one: 32768 x 4096 x 4096 254 us, so 202). B's scales are one tile (512 bytes) a word, or two.
#define MAXSIM_FP4_CP(TM, TOFF, SD, SOFF)                                         \
    "add.u32 t, " TM ", " TOFF ";\n\tadd.s64 s, " SD ", " SOFF ";\n\t"            \
    "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [t], s;\n\t"
#define MAXSIM_FP4_COPY(TEXT)                                                     \
    asm volatile("{\n\t.reg .pred e;\n\t.reg .b32 t;\n\t.reg .b64 s;\n\telect.sync _|e, 0xffffffff;\n\t" TEXT "}" ::"r"(sfa), "r"(sfb), \
                 "l"(fa), "l"(fb) : "memory")

// Scale tiles to tensor memory: four columns a tile, in all four lane quarters, on
// both CTAs from their own shared memory. Word j of A's goes to sfa + 4 j, of B's
// to sfb + 4 j, or 8 j and 8 j + 4.
template <int kWords, int kBTiles>
__device__ __forceinline__ void copy_scales(uint32_t sfa, uint32_t sfb, uint64_t fa, uint64_t fb) {
    if constexpr (kBTiles == 1) {
        MAXSIM_FP4_COPY(MAXSIM_FP4_CP("%0", "0", "%2", "0") MAXSIM_FP4_CP("%1", "0", "%3", "0")
                        MAXSIM_FP4_CP("%0", "4", "%2", "32") MAXSIM_FP4_CP("%1", "4", "%3", "32"));
        if constexpr (kWords == 4)
            MAXSIM_FP4_COPY(MAXSIM_FP4_CP("%0", "8", "%2", "64") MAXSIM_FP4_CP("%1", "8", "%3", "64")
                            MAXSIM_FP4_CP("%0", "12", "%2", "96") MAXSIM_FP4_CP("%1", "12", "%3", "96"));
    } else if constexpr (kWords == 4) {
        MAXSIM_FP4_COPY(MAXSIM_FP4_CP("%0", "0", "%2", "0") MAXSIM_FP4_CP("%1", "0", "%3", "0") MAXSIM_FP4_CP("%1", "4", "%3", "128")
                        MAXSIM_FP4_CP("%0", "4", "%2", "32") MAXSIM_FP4_CP("%1", "8", "%3", "32") MAXSIM_FP4_CP("%1", "12", "%3", "160")
                        MAXSIM_FP4_CP("%0", "8", "%2", "64") MAXSIM_FP4_CP("%1", "16", "%3", "64") MAXSIM_FP4_CP("%1", "20", "%3", "192")
                        MAXSIM_FP4_CP("%0", "12", "%2", "96") MAXSIM_FP4_CP("%1", "24", "%3", "96") MAXSIM_FP4_CP("%1", "28", "%3", "224"));
    } else {
        MAXSIM_FP4_COPY(MAXSIM_FP4_CP("%0", "0", "%2", "0") MAXSIM_FP4_CP("%1", "0", "%3", "0") MAXSIM_FP4_CP("%1", "4", "%3", "64")
                        MAXSIM_FP4_CP("%0", "4", "%2", "32") MAXSIM_FP4_CP("%1", "8", "%3", "32") MAXSIM_FP4_CP("%1", "12", "%3", "96"));
    }
}
#undef MAXSIM_FP4_CP
#undef MAXSIM_FP4_COPY

// Four K = 64 steps, 32 bytes of A's and B's rows a step (K-major, 128-byte
// swizzle), the first accumulating only if `accumulate` is nonzero. With blocks
// of 16 a step takes a scale word of each row, with blocks of 32 half a word
// (idesc_hi: the upper half).
#define MAXSIM_FP4_MMA(VEC, STEP, IDESC, AOFF, BOFF, PRED)                        \
    "add.s64 x, %1, " STEP ";\n\tadd.s64 y, %2, " STEP ";\n\tadd.u32 s, %4, " AOFF ";\n\tadd.u32 t, %5, " BOFF ";\n\t" \
    "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::" VEC " [%0], x, y, " IDESC ", [s], [t], " PRED ";\n\t"
#define MAXSIM_FP4_STAGE(TEXT)                                                    \
    asm volatile("{\n\t.reg .pred e, p0, pt;\n\t.reg .b32 s, t;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p0, %6, 0;\n\tsetp.eq.b32 pt, %6, %6;\n\t" \
                 "elect.sync _|e, 0xffffffff;\n\t" TEXT "}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(idesc_hi) \
                 : "memory")
template <int kWords, int kBTiles>
__device__ __forceinline__ void mma_stage(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t idesc_hi, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
    if constexpr (kWords == 4 && kBTiles == 1)
        MAXSIM_FP4_STAGE(MAXSIM_FP4_MMA("4X", "0", "%3", "0", "0", "p0") MAXSIM_FP4_MMA("4X", "2", "%3", "4", "4", "pt")
                         MAXSIM_FP4_MMA("4X", "4", "%3", "8", "8", "pt") MAXSIM_FP4_MMA("4X", "6", "%3", "12", "12", "pt"));
    else if constexpr (kWords == 4)
        MAXSIM_FP4_STAGE(MAXSIM_FP4_MMA("4X", "0", "%3", "0", "0", "p0") MAXSIM_FP4_MMA("4X", "2", "%3", "4", "8", "pt")
                         MAXSIM_FP4_MMA("4X", "4", "%3", "8", "16", "pt") MAXSIM_FP4_MMA("4X", "6", "%3", "12", "24", "pt"));
    else if constexpr (kBTiles == 1)
        MAXSIM_FP4_STAGE(MAXSIM_FP4_MMA("2X", "0", "%3", "0", "0", "p0") MAXSIM_FP4_MMA("2X", "2", "%7", "0", "0", "pt")
                         MAXSIM_FP4_MMA("2X", "4", "%3", "4", "4", "pt") MAXSIM_FP4_MMA("2X", "6", "%7", "4", "4", "pt"));
    else
        MAXSIM_FP4_STAGE(MAXSIM_FP4_MMA("2X", "0", "%3", "0", "0", "p0") MAXSIM_FP4_MMA("2X", "2", "%7", "0", "0", "pt")
                         MAXSIM_FP4_MMA("2X", "4", "%3", "4", "8", "pt") MAXSIM_FP4_MMA("2X", "6", "%7", "4", "8", "pt"));
}
#undef MAXSIM_FP4_MMA
#undef MAXSIM_FP4_STAGE

// v, loaded from tensor memory, is not used before the wait in front of this.
__device__ __forceinline__ void not_before(float (&v)[32]) {
    asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]),
                 "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]),
                 "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]));
    asm volatile("" : "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}

// The row scales' product s_x s_w comes first (its value does not depend on which
// of the operands is A), rounded to fp32's digits; one fma takes it to the sum and
// the bias. Where products of a warp's scales leave fp32's range, as those of rows
// of 2^-100 and of 2^100 may where the results do not, part of their exponents goes
// to the sums. What a scale asks of that: the exponents of its lowest and highest
// bits (biased by 127); zeros, infinities and NaN nothing.
__device__ __forceinline__ void scale_range(float s, int& low, int& high) {
    const uint32_t bits = __float_as_uint(s) & 0x7fffffffu;
    const int e = static_cast<int>(bits >> 23);
    if (bits == 0 || e == 255) return;
    low = min(low, e == 0 ? -22 : (bits & 0x7fffffu) ? e - 23 : e);
    high = max(high, e);
}
// 2^-62 <= |s| < 2^62: no product of two leaves the range.
__device__ __forceinline__ bool scale_near_one(float s) { return (__float_as_uint(s) & 0x7fffffffu) - (65u << 23) < (124u << 23); }
// s = m 2^k with 1 <= |m| < 2 (zeros, infinities and NaN: m = s, k = 0).
__device__ __forceinline__ void split_scale(float& s, int& k) {
    const float up = s * 0x1p24f;
    const bool tiny = fabsf(s) < 0x1p-126f;
    const uint32_t bits = __float_as_uint(tiny ? up : s), e = bits >> 23 & 255u;
    k = 0;
    if (e == 0 || e == 255u) return;
    k = static_cast<int>(e) - (tiny ? 151 : 127);
    s = __uint_as_float((bits & 0x807fffffu) | 0x3f800000u);
}
__device__ __forceinline__ float power_of_two(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }
// sum * m 2^k + bias, |m| < 4: m 2^k within fp32's range, the rest of 2^k goes to the sum
// (where it takes digits from it the result is far below fp32's least).
__device__ __forceinline__ float scale_sum(float sum, float m, int k, float bias) {
    const int near = max(-124, min(124, k)), rest = k - near, first = max(-126, min(127, rest));
    return __fmaf_rn(sum * power_of_two(first) * power_of_two(rest - first), m * power_of_two(near), bias);
}

// Every thread of every CTA of the cluster, whatever its warp's other threads do.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// One tile is 256 rows of A (128 on each CTA of a pair) x kTN rows of B (half on
// each). A is the larger operand: x, or w when kSwap.
//  * warps 0 and 3 bring stages of 256 values of K by TMA: its CTA's rows of A
//    and of B (128-byte swizzle) with the scale tiles of its rows of A and of all
//    the tile's rows of B, which both CTAs' MMA halves need. What lies outside the
//    operands reads as code 0 with scale 0. The bytes of both CTAs count on the
//    even one's barrier;
//  * warp 2 of the even CTA copies a stage's scales to tensor memory, warp 1
//    issues its MMAs (M = 256, N = kTN, K = 64);
//  * eight epilogue warps scale, add the bias, round once and store, as those of
//    linear_tile_kernel do.
// kRows16: rows of out start on 16-byte boundaries, and 16-bit ones end there.
// splits > 1 (few tiles): the pairs of a cluster share a tile's K; the others'
// sums pass to the first pair's shared memory and are added in their order.
// Measured: 32768 x 4096 x 4096 bf16, block 16, 176 us in short runs, 6.2 PFLOP/s;
// of a tile's 11,400 cycles (clock64) a stage takes 660, 512 of them MMAs, and 900
// pass until the one accumulator of 256 columns is free: 680 of the last MMAs, 330
// of the epilogue's reading it (whose 256-column tiles spill 40 bytes).
// 1048576 x 128 x 1024 f16: 129 us, 6.8 TB/s, HBM.
// 1 x 4096 x 4096: 7.6 us, latency.
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
            mbar_init(smem_u32(&ctl->full[s]), 2);  // even CTA: its two TMA warps, and all the pair's bytes
            mbar_init(smem_u32(&ctl->scales[s]), 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&ctl->acc_full[b]), 1);
            mbar_init(smem_u32(&ctl->acc_empty[b]), 16);  // eight warps of each CTA
        }
        mbar_init(smem_u32(&ctl->mma_done), 1);
        mbar_init(smem_u32(&ctl->copies_done), 1);
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

    // each branch runs under its own register budget
    if (warp < kFp4EpiWarp0) {
    regs_release<kFp4RegsCtl>();
    if (warp == 0 || warp == 3) {
        // ---------------------------------------------------------------- TMA: A with its scales, B with its scales
        if (lane == 0) {
            const bool is_a = warp == 0;
            const CUtensorMap* map = is_a ? &tm_a : &tm_b;
            const CUtensorMap* scale_map = is_a ? &tm_sfa : &tm_sfb;
            const uint32_t codes = smem_u32(is_a ? s_a : s_b), scales = smem_u32(is_a ? s_sfa : s_sfb);
            const uint32_t codes_step = is_a ? C::kA : C::kB, scales_step = is_a ? C::kSfa : C::kSfb;
            // both CTAs' loads count on the even one's barrier, which expects them all
            const uint32_t bars = map_shared_rank(smem_u32(&ctl->full[0]), even);
            const uint32_t bytes = 2 * (codes_step + static_cast<uint32_t>(words) * 512u * (is_a ? 1 : C::kBTiles));
            int32_t stage = 0;
            uint32_t phase = 0;
            int64_t issued = 0;
            bool ok = true;
            for (int64_t it = first; it < a.items && ok; it += step) {
                const int64_t row = it / a.tiles_b;
                // the codes' first row here, and the scales' first tile
                int32_t y = static_cast<int32_t>(row * kFp4TileM) + static_cast<int32_t>(rank) * 128, z = y >> 7;
                if (!is_a) {
                    y = static_cast<int32_t>(it - row * a.tiles_b) * kTN;
                    z = y >> 7;
                    y += static_cast<int32_t>(rank) * C::kBRows;
                }
                // The pairs that take one tile of A against all of B read its stages at the
                // same time, each fresh from HBM: what is next of A they bring to L2 before,
                // each its share.
                if (is_a && a.prefetch && it + step < a.items) {
                    const int64_t next = (it + step) / a.tiles_b;
                    const int32_t y2 = static_cast<int32_t>(next * kFp4TileM) + static_cast<int32_t>(rank) * 128;
                    for (int32_t kb = static_cast<int32_t>(it + step - next * a.tiles_b); kb < a.kb; kb += a.tiles_b) {
                        tma_prefetch_2d(map, kb * 128, y2);
                        tma_prefetch_3d(scale_map, 0, kb * words, y2 >> 7);
                    }
                }
                for (int32_t kb = kb0; kb < kb1; ++kb) {
                    if (!tile_wait(a, ctl, &ctl->empty[stage], phase ^ 1u)) { ok = false; break; }
                    if (rank == 0) mbar_arrive_expect_tx(smem_u32(&ctl->full[stage]), bytes);
                    tma_load_pair_2d(codes + stage * codes_step, map, bars + stage * 8, kb * 128, y);
                    tma_load_pair_3d(scales + stage * scales_step, scale_map, bars + stage * 8, 0, kb * words, z);
                    ++issued;
                    if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                }
            }
            if (ctl->abort) {  // the pair's copies still in flight land before the CTAs leave together
                const int64_t n = rank != 0 ? 0 : issued < C::kStages ? issued : C::kStages;
                for (int64_t i = 0; i < n; ++i) {
                    if (--stage < 0) { stage = C::kStages - 1; phase ^= 1u; }
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait(smem_u32(&ctl->full[stage]), phase) && global_timer_ns() - t0 < a.timeout_ns) {}
                }
                // the odd CTA cannot see its copies land: it allows them a thousand times what they take
                if (rank != 0 && issued > 0) {
                    const uint64_t t0 = global_timer_ns();
                    while (global_timer_ns() - t0 < a.timeout_ns / 500) {}
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
            const uint32_t sf0 = tmem + C::kAcc * kTN;
            const uint16_t both = static_cast<uint16_t>(3u << even);
            const bool b16 = a.block == 16;
            const uint32_t idesc = idesc_fp4(kFp4TileM, kTN, !b16, 0), idesc_hi = idesc_fp4(kFp4TileM, kTN, !b16, 2);
            int32_t buf = 0;
            uint32_t buf_phase = 0;
            for (int64_t it = first; it < a.items && ok; it += step) {
                // kTN = 64: the odd tiles' rows are the upper half of a scale tile
                const uint32_t sfb_off = kTN == 64 ? static_cast<uint32_t>((it % a.tiles_b) & 1) * 2u : 0u;
                if (!tile_wait_warp<true>(a, ctl, &ctl->acc_empty[buf], buf_phase ^ 1u)) break;
                tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>(buf * kTN);
                for (int32_t kb = kb0; kb < kb1; ++kb) {
                    // the scales are there, so the stage is (the warp that copied them has seen it land)
                    if (!tile_wait_warp<true>(a, ctl, &ctl->scales[stage], phase)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sfa = sf0 + static_cast<uint32_t>(stage * C::kSfCols), sfb = sfa + 16 + sfb_off;
                    const uint64_t da = a_desc + static_cast<uint64_t>((stage * C::kA) >> 4);
                    const uint64_t db = b_desc + static_cast<uint64_t>((stage * C::kB) >> 4);
                    const uint32_t acc = kb > kb0 ? 1u : 0u;
                    if (b16) mma_stage<4, C::kBTiles>(d, da, db, idesc, idesc_hi, sfa, sfb, acc);
                    else mma_stage<2, C::kBTiles>(d, da, db, idesc, idesc_hi, sfa, sfb, acc);
                    mma_commit_elect<2>(smem_u32(&ctl->empty[stage]), both);
                    if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                mma_commit_elect<2>(smem_u32(&ctl->acc_full[buf]), both);
                if (++buf == C::kAcc) { buf = 0; buf_phase ^= 1u; }
            }
            // every MMA issued above completes before the CTA leaves
            mma_commit_elect<2>(smem_u32(&ctl->mma_done), static_cast<uint16_t>(1u << even));
            if (lane == 0) {
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(smem_u32(&ctl->mma_done), 0) && global_timer_ns() - t0 < a.timeout_ns) {}
            }
            __syncwarp();
        }
    } else if (warp == 2) {
        // ---------------------------------------------------------------- scales (even CTA)
        if (rank == 0) {
            const uint64_t fa_desc = sdesc_scales(smem_u32(s_sfa)), fb_desc = sdesc_scales(smem_u32(s_sfb));
            const uint32_t sf0 = tmem + C::kAcc * kTN;
            int32_t stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t it = first; it < a.items && ok; it += step) {
                for (int32_t kb = kb0; kb < kb1; ++kb) {
                    // the MMAs of the stage's last use are done: its loads waited for them
                    if (!tile_wait_warp<true>(a, ctl, &ctl->full[stage], phase)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sfa = sf0 + static_cast<uint32_t>(stage * C::kSfCols);
                    const uint64_t fa = fa_desc + static_cast<uint64_t>((stage * C::kSfa) >> 4);
                    const uint64_t fb = fb_desc + static_cast<uint64_t>((stage * C::kSfb) >> 4);
                    if (words == 4) copy_scales<4, C::kBTiles>(sfa, sfa + 16, fa, fb);
                    else copy_scales<2, C::kBTiles>(sfa, sfa + 16, fa, fb);
                    mma_commit_elect<2>(smem_u32(&ctl->scales[stage]), static_cast<uint16_t>(1u << even));
                    if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                }
            }
            // every copy issued above completes before the CTA leaves
            mma_commit_elect<2>(smem_u32(&ctl->copies_done), static_cast<uint16_t>(1u << even));
            if (lane == 0) {
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(smem_u32(&ctl->copies_done), 0) && global_timer_ns() - t0 < a.timeout_ns) {}
            }
            __syncwarp();
        }
    }
    if (a.splits > 1) {  // the epilogue warps' two meetings
        cluster_arrive();
        cluster_wait();
        cluster_arrive();
        cluster_wait();
    }
    } else {
        regs_claim<kFp4RegsEpi>();
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
            float sa = scale_a && in_a ? __ldg(scale_a + ra0 + lane) : 1.f;
            float bias_a = kSwap && a.l.bias && in_a ? __ldg(a.l.bias + ra0 + lane) : 0.f;
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
            const uint32_t src0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * kCols);
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
            if (a.splits == 1) {
                if (!tile_wait_warp(a, ctl, &ctl->acc_full[buf], buf_phase)) break;
                tc_fence_after();
            }
            const uint32_t src = src0 + static_cast<uint32_t>(buf * kTN);
            // all of the lane's sums, then the accumulator is handed back
            float v[kChunks][32];
#pragma unroll
            for (int c = 0; c < kChunks; ++c) tmem_ld32(src + c * 32, v[c]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < kChunks; ++c) not_before(v[c]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(map_shared_rank(smem_u32(&ctl->acc_empty[buf]), even));
            if (a.splits > 1) {
                for (int32_t s = 0; s + 1 < a.splits; ++s)
#pragma unroll
                    for (int i = 0; i < kCols; ++i) v[i / 32][i % 32] += parts[s * (kTN * 128) + i * 128];
            }
            bool plain = scale_near_one(sa);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) plain = plain && scale_near_one(sb[c]);
            plain = __all_sync(0xffffffffu, plain);
            if (!plain) {
                // all products in range, and those of powers of two exact (zero rows have 2^-126)?
                int low_a = 127, high_a = 127, low_b = 127, high_b = 127;
                scale_range(sa, low_a, high_a);
#pragma unroll
                for (int c = 0; c < kChunks; ++c) scale_range(sb[c], low_b, high_b);
                plain = __reduce_min_sync(0xffffffffu, low_a) + __reduce_min_sync(0xffffffffu, low_b) >= 254 - 149 &&
                        __reduce_max_sync(0xffffffffu, high_a) + __reduce_max_sync(0xffffffffu, high_b) <= 254 + 126;
            }
            if (!plain) {  // results in place of the sums
                int ka, kb[kChunks];
                split_scale(sa, ka);
#pragma unroll
                for (int c = 0; c < kChunks; ++c) split_scale(sb[c], kb[c]);
#pragma unroll
                for (int i = 0; i < kCols; ++i) {
                    const int c = i / 32;
                    const float m = sa * __shfl_sync(0xffffffffu, sb[c], i % 32), more = kSwap ? bias_a : __shfl_sync(0xffffffffu, bias[c], i % 32);
                    v[c][i % 32] = scale_sum(v[c][i % 32], m, ka + __shfl_sync(0xffffffffu, kb[c], i % 32), more);
                }
                sa = 1.f;
                bias_a = 0.f;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    sb[c] = 1.f;
                    bias[c] = 0.f;
                    if constexpr (kHold) {
                        tab[c * 32 + lane] = 1.f;
                        if constexpr (!kSwap) tab[kCols + c * 32 + lane] = 0.f;
                    }
                }
                __syncwarp();
            }
            const float2 sa2 = make_float2(sa, sa);
            if constexpr (kHold) {
#pragma unroll
                for (int i = 0; i < kCols; i += 4) {
                    const float* u = v[i / 32] + i % 32;
                    const float4 s4 = *reinterpret_cast<const float4*>(tab + i);
                    const float4 b4 = kSwap ? make_float4(bias_a, bias_a, bias_a, bias_a) : *reinterpret_cast<const float4*>(tab + kCols + i);
                    const float2 lo = fma2(make_float2(u[0], u[1]), mul2(make_float2(s4.x, s4.y), sa2), make_float2(b4.x, b4.y));
                    const float2 hi = fma2(make_float2(u[2], u[3]), mul2(make_float2(s4.z, s4.w), sa2), make_float2(b4.z, b4.w));
                    held[i / 32][i % 32 / 2] = pack2<T>(lo.x, lo.y);
                    held[i / 32][i % 32 / 2 + 1] = pack2<T>(hi.x, hi.y);
                }
            }
            if (++buf == C::kAcc) { buf = 0; buf_phase ^= 1u; }
            if constexpr (kHold) {
                store_held<T, kCols, kSwap, kTma>(held, stage, out, ld, ra0, rb0, a.rows_b, row_n, &tm_out);
            } else {
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const int64_t rb = rb0 + c * 32;
                    if (row_n == 0 || rb >= a.rows_b) break;
                    if constexpr (kSwap) {
                        const int n = static_cast<int>(min(static_cast<int64_t>(32), a.rows_b - rb));
                        float* p = out + rb * ld + ra0 + lane;
#pragma unroll
                        for (int i = 0; i < 32; ++i, p += ld) {
                            const float y = __fmaf_rn(v[c][i], __shfl_sync(0xffffffffu, sb[c], i) * sa, bias_a);
                            if (i < n && in_a) *p = y;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<float4*>(stage + staged(lane, i)) =
                                make_float4(v[c][4 * i], v[c][4 * i + 1], v[c][4 * i + 2], v[c][4 * i + 3]);
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
                                const float xs = __shfl_sync(0xffffffffu, sa, 4 * i + (lane >> 3));  // of the row
                                if (4 * i + (lane >> 3) < row_n)
                                    store4(out + at, n, __fmaf_rn(y.x, ws[0] * xs, bs[0]), __fmaf_rn(y.y, ws[1] * xs, bs[1]),
                                           __fmaf_rn(y.z, ws[2] * xs, bs[2]), __fmaf_rn(y.w, ws[3] * xs, bs[3]));
                            }
                        } else {  // rows off their 16-byte boundaries: a row at a time, a lane per column
                            const bool in_b = rb + lane < a.rows_b;
                            const uint8_t* from = stage + (lane & 3) * 4;
                            int64_t at = ra0 * ld + rb + lane;
#pragma unroll 8
                            for (int r = 0; r < row_n; ++r, at += ld) {
                                const float y = *reinterpret_cast<const float*>(from + staged(r, lane >> 2));
                                const float f = sb[c] * __shfl_sync(0xffffffffu, sa, r);
                                if (in_b) out[at] = __fmaf_rn(y, f, bias[c]);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
        }
        if (kTma && lane == 0) bulk_wait();
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
