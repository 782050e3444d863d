// out[m, n] = (sum_k x[m, k] w[n, k]) * x_scale[m] * w_scale[n] + bias[n] for
// 8-bit integers x [M, K] and w [N, K].
//
// sm_103a has no 8-bit integer kind among its tcgen05 MMAs, and mma.sync's
// 8-bit integer form was measured at 150 TOP/s, a quarter of the f16 form's
// 605 TFLOP/s. So both kernels widen the integers to binary16 on the SM, next
// to the tensor cores: |v| <= 128 is exact there, a product of two is exact in
// fp32, and a sum of up to 1,024 products (2^24) is too; longer ones are added
// as integers (16-bit outputs of the tile kernel apart, see parts_needed).
//
//  * linear_few_kernel (few tokens, and small products of any shape): bound by
//    the bytes of w, each read once per 32 tokens, or by its launch.
//  * linear_tile_kernel (everything else): tcgen05 MMAs of 256-row tiles on CTA
//    pairs, bound by the tensor pipe, or by the bytes of the larger operand
//    where the other one is narrow.
#pragma once

#include <cstdint>

#include "head_kernels.cuh"
#include "ptx.cuh"

namespace maxsim {

struct LinearArgs {
    const int8_t* x;
    const int8_t* w;
    int64_t ld_x, ld_w, ld_out;
    const float* x_scale;
    const float* w_scale;
    const float* bias;  // NULL = none
    void* out;
    int32_t M, N, K;
};

// A dependent launch may begin while the kernel before it still runs: it then
// waits, where it reads that kernel's results, for all of it to be done.
__device__ __forceinline__ void begin_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// 16 bytes of a row from k on, zero from K on, where rows start anywhere:
// aligned words shifted into place. The words may hold bytes of neighbouring
// rows, but none outside the operand's [base, end): its first and last bytes
// are loaded one by one.
__device__ __forceinline__ uint4 load16_any(const int8_t* row, int32_t k, int32_t K, const int8_t* base, const int8_t* end) {
    uint32_t w[4] = {0, 0, 0, 0};
    const int n = K - k;
    if (n <= 0) return make_uint4(0, 0, 0, 0);
    const int8_t* p = row + k;
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 3);
    const int8_t* first = p - shift;
    if (first >= base && first + 20 <= end) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(first);
        uint32_t v[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) v[i] = __ldg(q + i);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = __funnelshift_r(v[i], v[i + 1], shift * 8);
            const int left = n - 4 * i;  // bytes of this word that exist
            if (left < 4) w[i] &= left <= 0 ? 0u : 0xffffffffu >> (32 - 8 * left);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (e < n) w[e >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(__ldg(p + e))) << ((e & 3) * 8);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Operands laid out once for the tile kernel.
struct PrepJob {
    const int8_t* src;
    void* dst;
    int64_t rows, ld_src;
    int direct;  // rows are whole 16-byte pieces on 16-byte boundaries
};
struct PrepArgs {
    PrepJob copy;   // to rows of k_pad bytes (A, where its rows are off their 16-byte boundaries)
    PrepJob widen;  // to rows of k_pad halves (the tile kernel's smaller operand)
    int32_t K, k_pad;  // k_pad a multiple of 16: the tail is zero
};

__device__ __forceinline__ uint4 load_row16(const PrepJob& j, int64_t r, int32_t k, int32_t K) {
    const int8_t* row = j.src + r * j.ld_src;
    if (j.direct) return __ldg(reinterpret_cast<const uint4*>(row + k));
    return load16_any(row, k, K, j.src, j.src + (j.rows - 1) * j.ld_src + K);
}

// One pass, bound by its bytes: 4096 x 4096 widened in about 8 us.
static __global__ void __launch_bounds__(256) linear_prep_kernel(const PrepArgs a) {
    begin_dependents();
    const int32_t per_row = a.k_pad >> 4;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x, n1 = a.widen.rows * per_row,
                  n2 = n1 + a.copy.rows * per_row;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n2; i += step) {
        const PrepJob& j = i < n1 ? a.widen : a.copy;
        const int64_t at = i < n1 ? i : i - n1;
        const int64_t r = at / per_row;
        const int32_t k = static_cast<int32_t>(at - r * per_row) << 4;
        const uint4 v = load_row16(j, r, k, a.K);
        if (i < n1) {
            uint4* to = reinterpret_cast<uint4*>(static_cast<__half*>(j.dst) + r * a.k_pad + k);
            to[0] = i8x8_to_f16x8(v.x, v.y);
            to[1] = i8x8_to_f16x8(v.z, v.w);
        } else {
            *reinterpret_cast<uint4*>(static_cast<int8_t*>(j.dst) + r * a.k_pad + k) = v;
        }
    }
}

// ---------------------------------------------------------------- few tokens, small products

__device__ __forceinline__ void mma_m16n8k16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes to 16 halves: h[i] holds elements 2i and 2i + 1.
__device__ __forceinline__ void widen16(uint4 v, uint32_t (&h)[8]) {
    const uint4 lo = i8x8_to_f16x8(v.x, v.y), hi = i8x8_to_f16x8(v.z, v.w);
    h[0] = lo.x; h[1] = lo.y; h[2] = lo.z; h[3] = lo.w;
    h[4] = hi.x; h[5] = hi.y; h[6] = hi.z; h[7] = hi.w;
}

constexpr int kFewWarps = 16;  // most warps of a block

// kWhole: rows are whole 16-byte pieces on 16-byte boundaries.
template <bool kWhole>
__device__ __forceinline__ uint4 load16(const int8_t* row, int32_t k, int32_t K, const int8_t* base, const int8_t* end) {
    if constexpr (kWhole) return k < K ? __ldg(reinterpret_cast<const uint4*>(row + k)) : make_uint4(0, 0, 0, 0);
    else return load16_any(row, k, K, base, end);
}

// A block owns 16 channels and up to 8 * kTiles tokens (blockIdx.y); its warps
// take runs of 64-wide chunks of K. A lane reads 16 consecutive bytes of two
// channels (w is the MMA's 16-row operand) and of one token of each 8-token
// tile: lane t of a row then holds k = 16 t .. 16 t + 15 instead of the
// fragment's own columns, in both operands alike, so the sum over k is the
// same and every load is 16 bytes wide; the loads of the next chunks are in
// flight while one is widened. After 16 chunks of a warp (1,024
// products, exact in fp32) the sums move to 32-bit integers, and the warps'
// sums are added as integers in shared memory: exact, in any order. Bound by the
// bytes of w in flight (1 x 16384 x 16384: 51 us, 5.2 TB/s), by the widening of
// the tokens, which every block repeats, as they get more (32 x 4096 x 4096:
// 8.3 us, and 4.6 with one), and by its launch when small (32 x 128 x 1024:
// 3.8 us).
template <typename T, int kTiles, bool kWhole>
__global__ void __launch_bounds__(kFewWarps * 32) linear_few_kernel(const LinearArgs a) {
    constexpr int kAhead = !kWhole ? 1 : kTiles == 2 ? 4 : 2;  // chunks whose loads are in flight
    __shared__ int s_sum[16][8 * kTiles + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16, m0 = static_cast<int64_t>(blockIdx.y) * (8 * kTiles);
    for (int i = threadIdx.x; i < 16 * (8 * kTiles + 1); i += blockDim.x) (&s_sum[0][0])[i] = 0;
    __syncthreads();
    // rows past the ends read the last row; what they give is not stored
    const int8_t* w0 = a.w + min(n0 + g, static_cast<int64_t>(a.N) - 1) * a.ld_w;
    const int8_t* w1 = a.w + min(n0 + g + 8, static_cast<int64_t>(a.N) - 1) * a.ld_w;
    const int8_t* xr[kTiles];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) xr[j] = a.x + min(m0 + 8 * j + g, static_cast<int64_t>(a.M) - 1) * a.ld_x;
    const int8_t* x_end = a.x + (static_cast<int64_t>(a.M) - 1) * a.ld_x + a.K;
    const int8_t* w_end = a.w + (static_cast<int64_t>(a.N) - 1) * a.ld_w + a.K;
    // this warp's run of chunks, and where its values end
    const int32_t chunks = (a.K + 63) >> 6, run = (chunks + warps - 1) / warps;
    const int32_t c0 = warp * run, c1 = min(chunks, c0 + run), k_end = min(a.K, c1 << 6);
    uint4 wv[kAhead][2], xv[kAhead][kTiles];
    auto load = [&](int slot, int32_t chunk) {
        const int32_t k = (chunk << 6) + 16 * t;
        wv[slot][0] = load16<kWhole>(w0, k, k_end, a.w, w_end);
        wv[slot][1] = load16<kWhole>(w1, k, k_end, a.w, w_end);
#pragma unroll
        for (int j = 0; j < kTiles; ++j) xv[slot][j] = load16<kWhole>(xr[j], k, k_end, a.x, x_end);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i, c0 + i);
    int sum[kTiles][4] = {};
    float acc[kTiles][4] = {};
#pragma unroll 1
    for (int32_t c = c0; c < c1; c += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            uint32_t wa[8], wb[8];
            widen16(wv[i][0], wa);
            widen16(wv[i][1], wb);
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                uint32_t xb[8];
                widen16(xv[i][j], xb);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    mma_m16n8k16(acc[j], wa[2 * s], wb[2 * s], wa[2 * s + 1], wb[2 * s + 1], xb[2 * s], xb[2 * s + 1]);
            }
            load(i, c + i + kAhead);
        }
        if (((c - c0 + kAhead) & 15) == 0 || c + kAhead >= c1) {
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sum[j][e] += __float2int_rn(acc[j][e]);
                    acc[j][e] = 0.f;
                }
        }
    }
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) atomicAdd(&s_sum[g + (e & 2) * 4][8 * j + 2 * t + (e & 1)], sum[j][e]);
    __syncthreads();
    const int tokens = static_cast<int>(min(a.M - m0, static_cast<int64_t>(8 * kTiles)));
    for (int i = threadIdx.x; i < 16 * tokens; i += blockDim.x) {
        const int m = i >> 4, n = i & 15;
        if (n0 + n < a.N) {
            float v = static_cast<float>(s_sum[n][m]) * a.x_scale[m0 + m] * a.w_scale[n0 + n];
            if (a.bias) v += a.bias[n0 + n];
            static_cast<T*>(a.out)[(m0 + m) * a.ld_out + n0 + n] = from_f32<T>(v);
        }
    }
}

// ---------------------------------------------------------------- many tokens

constexpr int kTileM = 256;            // rows of A per tile: 128 on each CTA of a pair
constexpr int kTileK = 128;            // values of K per block
constexpr int kExactBlocks = 8;        // blocks whose sums are exact in fp32: 1,024 products of at most 2^14
constexpr int kTileRing = 4;           // blocks ready for the MMA: A in tensor memory, B in shared memory
constexpr int kTileBWarp = 2, kWidenWarp0 = 4, kTileEpiWarp0 = 12;
constexpr int kTileThreads = 640;      // warp 0 TMA of A, warp 1 MMA, warp 2 TMA of B, warps 4-11 widen, 12-19 epilogue
constexpr int kTileMaxStages8 = 8;
// Registers per thread: the launch gives every thread kTileRegs; warps 0-3 and
// the widening warps hand registers to the epilogue warps, which hold a
// tile's rounded outputs until they are stored. 16-bit outputs, which are held,
// get 8 more than others (1048576 x 64 x 1024 f16 195 -> 189 us; f32 would lose a
// little, 4096 x 4096 x 4096 102.5 -> 103.4). What is spilled, 44 to 76 bytes of
// most variants, is the control and the widening warps' (compiled with 80
// registers for the former, or 96 for the latter, half of it goes; with 200
// for the epilogue, next to nothing).
constexpr int kTileRegs = 96, kTileRegsCtl = 48;
__host__ __device__ constexpr int tile_regs_epi(bool held) { return held ? 144 : 136; }
__host__ __device__ constexpr int tile_regs_widen(bool held) { return 216 - tile_regs_epi(held); }
static_assert(kTileRegsCtl * 128 + 216 * 256 <= kTileRegs * kTileThreads, "register split");
constexpr int kTileStage = 4096;       // staging of an epilogue warp: 32 x 32 sums
constexpr uint32_t kTileACol = 256;    // tensor memory: accumulators in columns 0-255, the ring's A blocks above
constexpr int kTileStatusTimeout = 4;  // MAXSIM_ERR_TIMEOUT

// kKeepB: B is one tile of rows for all tiles of A, and its blocks stay in shared memory.
template <int kTN, bool kKeepB>
struct TileCfg {
    static constexpr int kA8 = 128 * kTileK;           // 8-bit block of A: this CTA's 128 rows
    static constexpr int kBRows = kTN / 2;             // rows of B per CTA
    static constexpr int kBAtom = kBRows * 128;        // 64 halves of every row
    static constexpr int kB16 = 2 * kBAtom;
    // even: each widening warpgroup then always meets the same stages, and
    // sees every phase of their barriers
    static constexpr int kStages8 = kTN == 256 || kKeepB ? 4 : 8;
    static constexpr int kStagesB = !kKeepB ? kTileRing : kTN == 128 ? 8 : 16;  // kKeepB: the most blocks of K
    static constexpr int kAcc = kTN == 256 ? 1 : 2;    // accumulator buffers
};

// Whether 32-bit results (f32 outputs, and the integer sums of slices) of `blocks`
// blocks of K are summed in parts. Past kExactBlocks an fp32 accumulator may
// round; the epilogue then takes what it holds and adds the parts without loss,
// as 32-bit integers, or two of them as floats (the one rounding of an exact
// sum). Tiles of 256 columns have no registers for those sums: 32768 x 4096 x
// 4096 f32 takes 700 us in tiles of 128, and 585 in one accumulator of 256
// columns; shorter or narrower products lose 2 to 11 %. 16-bit outputs stay in one
// accumulator (528 us; tiles of 128 columns without parts take 644): past 2^24
// a step of 16 products may lose 2^-23 of the partial sum, for sums of one
// sign up to K = 16,384 at most a quarter of an f16 output's rounding.
constexpr bool parts_needed(int32_t blocks) { return blocks > kExactBlocks; }

struct TileArgs {
    LinearArgs l;
    int32_t* partial;   // [slices, M, N] integer sums (T = int32_t)
    int64_t items;      // tiles * slices, < 2^32 (the divisions of short items are worth 32 bits)
    int32_t rows_a;     // rows of A (tokens, or channels when swapped)
    int32_t rows_b;
    int32_t tiles_b;
    int32_t slices;     // parts of K
    int32_t kb;         // blocks of K
    int32_t kb_slice;   // blocks per slice
    int32_t kb_part;    // kParts: blocks per part, of one size but for a slice's last one
    int a_prepared;     // A too was laid out by linear_prep_kernel
    int* status;
    uint64_t timeout_ns;
};

struct alignas(16) TileCtl {
    uint64_t full8[kTileMaxStages8], empty8[kTileMaxStages8];
    uint64_t b_full[kTileRing], ready[kTileRing], freed[kTileRing];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    volatile int32_t abort;
};

template <int kTN, bool kKeepB>
constexpr size_t tile_smem_bytes() {
    using C = TileCfg<kTN, kKeepB>;
    return 1024 + static_cast<size_t>(C::kStages8) * C::kA8 + C::kStagesB * C::kB16 + 8 * kTileStage + sizeof(TileCtl);
}

// Bounded wait of a thread: gives up after the limit (recorded in the device
// status word) or when another role of the CTA has.
template <bool kCluster = false>
__device__ __forceinline__ bool tile_wait(const TileArgs& a, TileCtl* ctl, uint64_t* bar_ptr, uint32_t parity) {
    const uint32_t bar = smem_u32(bar_ptr);
    if (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (ctl->abort) return false;
            if (global_timer_ns() - t0 > a.timeout_ns) {
                ctl->abort = 1;
                atomicCAS(a.status, 0, kTileStatusTimeout);
                return false;
            }
        }
    }
}

template <bool kCluster = false>
__device__ __forceinline__ bool tile_wait_warp(const TileArgs& a, TileCtl* ctl, uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, tile_wait<kCluster>(a, ctl, bar, parity));
}

// 32 registers into 32 consecutive columns of this thread's tensor-memory lane.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}

// Waits for this thread's tensor-memory loads; v, loaded by one of them, is not used before.
__device__ __forceinline__ void tmem_wait_ld16(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four K = 16 steps into d with A in tensor memory (8 columns a step) and B in
// shared memory (K-major, 128-byte swizzle: 32 bytes a step), from the elected
// lane. The first step accumulates only if `accumulate` is nonzero.
__device__ __forceinline__ void mma_chain4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p0, pt;\n\t.reg .b64 b1, b2, b3;\n\t.reg .b32 a1, a2, a3;\n\t"
        "setp.ne.b32 p0, %4, 0;\n\t"
        "setp.eq.b32 pt, %4, %4;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a1], b1, %3, pt;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a2], b2, %3, pt;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a3], b3, %3, pt;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

struct TileItem {
    int64_t a0, b0;  // this CTA's first row of A, the tile's first row of B
    int32_t kb0, kb1;
    int32_t slice;
};

template <int kTN>
__device__ __forceinline__ TileItem tile_item(const TileArgs& a, uint32_t item, uint32_t rank) {
    TileItem t;
    const uint32_t tile = item / static_cast<uint32_t>(a.slices), row = tile / static_cast<uint32_t>(a.tiles_b);
    t.slice = static_cast<int32_t>(item - tile * static_cast<uint32_t>(a.slices));
    t.a0 = static_cast<int64_t>(row) * kTileM + rank * 128;
    t.b0 = static_cast<int64_t>(tile - row * static_cast<uint32_t>(a.tiles_b)) * kTN;
    t.kb0 = t.slice * a.kb_slice;
    t.kb1 = min(a.kb, t.kb0 + a.kb_slice);
    return t;
}

// a * b and a * b + c of two values in one instruction, each rounded once.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    mul2_rn(a.x, a.y, b.x, b.y);
    return a;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// Integer sums pass the epilogue as their bits.
template <>
__device__ __forceinline__ int32_t from_f32<int32_t>(float v) { return __float_as_int(v); }

// Byte of the 16-byte piece c of row r in a warp's staging tile [32][32] of
// 4-byte values: 32 lanes that write one piece each of their own row, or read
// the eight pieces of four rows, meet no bank twice.
__device__ __forceinline__ uint32_t staged(int r, int c) { return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4)); }

// The same piece in the box of a TMA store of 32 rows x 32 * kJoin 16-bit values
// (rows of 128 or 64 bytes, swizzled as wide): no bank twice either.
template <int kJoin>
__device__ __forceinline__ uint32_t boxed(int r, int c) {
    if constexpr (kJoin == 2) return staged(r, c);
    else return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// Four consecutive 32-bit elements from p (16-byte aligned) on, of which the first n exist.
template <typename T>
__device__ __forceinline__ void store4(T* p, int n, float a, float b, float c, float d) {
    static_assert(sizeof(T) == 4, "one 16-byte store");
    if (n >= 4) {
        alignas(16) T o[4] = {from_f32<T>(a), from_f32<T>(b), from_f32<T>(c), from_f32<T>(d)};
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(o);
    } else {
        if (n > 0) p[0] = from_f32<T>(a);
        if (n > 1) p[1] = from_f32<T>(b);
        if (n > 2) p[2] = from_f32<T>(c);
        if (n > 3) p[3] = from_f32<T>(d);
    }
}

// One tile is 256 rows of A (128 on each CTA of a pair) x kTN rows of B. A is
// the larger operand (x, or w when kSwap) and stays 8-bit until it is on the
// SM; B, the smaller one, was widened to halves in device memory once for all
// tiles (linear_prep_kernel).
//  * TMA brings 128-byte-wide blocks of A's rows into a ring of 8-bit stages
//    and blocks of B (each CTA half of the tile's rows) into a ring of operand
//    stages (128-byte swizzle; rows and columns past the ends read as 0);
//  * eight widening warps, alternating blocks by warpgroup, turn A's rows into
//    halves in tensor memory: a thread owns a row, as an MMA with A in tensor
//    memory wants it. Widened into shared memory, A would be written and read
//    there once more, which with B's traffic takes more time than the MMA;
//  * one warp of the even CTA issues tcgen05.mma.cta_group::2 (M = 256, N =
//    kTN, K = 16);
//  * eight epilogue warps scale, add the bias, round once and store.
// What a widening warp hands to the MMA is in tensor memory (ordered by
// tcgen05.fence::before_thread_sync), and what the odd CTA reports of B was
// written by TMA (observed on b_full), so these arrivals on the even CTA's
// barriers release at CTA scope. A cluster-scope release took a warp 800 to
// 2,000 cycles per block (32768 x 4096 x 4096: 751 us, and 609 us without).
// Narrow tiles are bound by what the SMs read from L2 (16384 x 128 x 4096: a
// block of A and of B in 650 cycles, 11 TB/s over all SMs, whatever the MMAs and
// the widening took). Where B is a single tile of rows and fits, as a head's
// weights do, it is loaded once and kept (kKeepB).
// kRows16: rows of out (of the sums) start on 16-byte boundaries, and those of
// 16-bit outputs end there. (Both ways of storing in one kernel cost this one
// 3 to 8 %.)
// A tile's K may be cut into slices (few tiles, long K): each slice then
// writes its integer sums (T = int32_t), and linear_join_kernel adds them.
// kParts: 32-bit results of more than kExactBlocks blocks of K (parts_needed).
// Measured with the preparation: 32768 x 4096 x 4096 in 525 us, 2.09 PFLOP/s
// (tensor pipe 87 % active; 584 to 605 us, 1.8 to 1.9 PFLOP/s, once the power limit
// holds the clock), 1048576 x 128 x 1024 in 210 us, 6.4 TB/s (HBM), 2048 x 4096 x 1024
// in 18.1 us (two rounds of tiles, the last one's stores).
template <typename T, int kTN, bool kSwap, bool kKeepB, bool kRows16, bool kParts>
__global__ void __launch_bounds__(kTileThreads, 1)
linear_tile_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ CUtensorMap tm_out, const TileArgs a) {
    using C = TileCfg<kTN, kKeepB>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* s8 = smem;
    uint8_t* s16 = smem + C::kStages8 * C::kA8;
    uint8_t* s_out = s16 + C::kStagesB * C::kB16;
    TileCtl* ctl = reinterpret_cast<TileCtl*>(s_out + 8 * kTileStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    constexpr bool kSums = std::is_same_v<T, int32_t>;
    static_assert(!kParts || (sizeof(T) == 4 && kTN <= 128), "registers for the parts' sums");
    if constexpr (kSums) begin_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages8; ++s) {
            mbar_init(smem_u32(&ctl->full8[s]), 1);
            mbar_init(smem_u32(&ctl->empty8[s]), 4);
        }
        for (int r = 0; r < kTileRing; ++r) {
            // its own TMA; kKeepB, even CTA: and the odd CTA's report
            mbar_init(smem_u32(&ctl->b_full[r]), kKeepB && rank == 0 ? 2 : 1);
            // even CTA: four widening warps of each CTA, its own TMA of B, the odd CTA's report of B
            mbar_init(smem_u32(&ctl->ready[r]), kKeepB ? 8 : 10);
            mbar_init(smem_u32(&ctl->freed[r]), 1);
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
    }
    if (warp == 1) {
        tmem_alloc<2>(smem_u32(&ctl->tmem_base), 512);
        tmem_relinquish<2>();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // barriers of both CTAs exist before any remote arrival
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;

    // each branch runs under its own register budget
    if (warp < kWidenWarp0) {
    regs_release<kTileRegsCtl>();
    if (warp == 0 || warp == kTileBWarp) {
        // ------------------------------------------------------------ TMA
        if (lane == 0) {
            const bool is_a = warp == 0;
            if (!is_a || a.a_prepared) wait_for_previous();
            const int depth = is_a ? C::kStages8 : kTileRing;
            // the even CTA's B lands on the barrier that its MMA warp waits for
            uint64_t* full = is_a ? ctl->full8 : rank == 0 && !kKeepB ? ctl->ready : ctl->b_full;
            uint64_t* empty = is_a ? ctl->empty8 : ctl->freed;
            int32_t stage = 0;
            uint32_t phase = 0;
            int64_t issued = 0;
            bool ok = true;
            if (kKeepB && !is_a && first < a.items) {  // every block once
                const uint32_t bar = smem_u32(&ctl->b_full[0]);
                mbar_arrive_expect_tx(bar, static_cast<uint32_t>(a.kb * C::kB16));
                for (int32_t kb = 0; kb < a.kb; ++kb) {
                    const uint32_t dst = smem_u32(s16 + kb * C::kB16);
                    tma_load_2d(dst, &tm_b, bar, kb * kTileK, static_cast<int32_t>(rank) * C::kBRows);
                    tma_load_2d(dst + C::kBAtom, &tm_b, bar, kb * kTileK + 64, static_cast<int32_t>(rank) * C::kBRows);
                }
                ++issued;
                stage = 1;
            }
            for (int64_t it = first; it < a.items && ok && (is_a || !kKeepB); it += step) {
                const TileItem t = tile_item<kTN>(a, it, rank);
                for (int32_t kb = t.kb0; kb < t.kb1; ++kb) {
                    if (!tile_wait(a, ctl, &empty[stage], phase ^ 1u)) { ok = false; break; }
                    const uint32_t bar = smem_u32(&full[stage]);
                    if (is_a) {
                        mbar_arrive_expect_tx(bar, C::kA8);
                        tma_load_2d(smem_u32(s8 + stage * C::kA8), &tm_a, bar, kb * kTileK, static_cast<int32_t>(t.a0));
                    } else {
                        const int32_t row = static_cast<int32_t>(t.b0) + static_cast<int32_t>(rank) * C::kBRows;
                        const uint32_t dst = smem_u32(s16 + stage * C::kB16);
                        mbar_arrive_expect_tx(bar, C::kB16);
                        tma_load_2d(dst, &tm_b, bar, kb * kTileK, row);
                        tma_load_2d(dst + C::kBAtom, &tm_b, bar, kb * kTileK + 64, row);
                    }
                    ++issued;
                    if (++stage == depth) { stage = 0; phase ^= 1u; }
                }
            }
            if (ctl->abort) {  // the copies still in flight land before the CTA leaves
                const int64_t n = issued < depth ? issued : depth;
                for (int64_t i = 0; i < n; ++i) {
                    if (--stage < 0) { stage = depth - 1; phase ^= 1u; }
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait(smem_u32(&full[stage]), phase) && global_timer_ns() - t0 < a.timeout_ns) {}
                }
            }
        }
    } else if (warp == 1) {
        int32_t ring = 0;
        uint32_t ring_phase = 0;
        bool ok = true;
        if (rank == 0) {
            // ------------------------------------------------------------ MMA (even CTA)
            constexpr uint32_t idesc = idesc_f16_f32(0, kTileM, kTN);
            const uint64_t b0 = sdesc_k_sw128(smem_u32(s16));
            int32_t buf = 0;
            uint32_t buf_phase = 0;
            if (kKeepB && first < a.items) ok = tile_wait_warp<true>(a, ctl, &ctl->b_full[0], 0);
            for (int64_t it = first; it < a.items && ok; it += step) {
                const TileItem t = tile_item<kTN>(a, it, rank);
                int32_t s0 = t.kb0;
                do {  // a run of blocks that are summed in one accumulator
                    const int32_t s1 = kParts ? min(t.kb1, s0 + a.kb_part) : t.kb1;
                    if (!tile_wait_warp<true>(a, ctl, &ctl->acc_empty[buf], buf_phase ^ 1u)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t d = tmem + static_cast<uint32_t>(buf * kTN);
                    for (int32_t kb = s0; kb < s1; ++kb) {
                        if (!tile_wait_warp<true>(a, ctl, &ctl->ready[ring], ring_phase)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t at = tmem + kTileACol + static_cast<uint32_t>(ring * 64);
                        const uint64_t b = b0 + static_cast<uint64_t>(((kKeepB ? kb : ring) * C::kB16) >> 4);
                        mma_chain4_ts(d, at, b, idesc, kb > s0 ? 1u : 0u);
                        mma_chain4_ts(d, at + 32, b + (C::kBAtom >> 4), idesc, 1u);
                        mma_commit_elect<2>(smem_u32(&ctl->freed[ring]));
                        if (++ring == kTileRing) { ring = 0; ring_phase ^= 1u; }
                    }
                    if (!ok) break;
                    mma_commit_elect<2>(smem_u32(&ctl->acc_full[buf]));
                    if (++buf == C::kAcc) { buf = 0; buf_phase ^= 1u; }
                    s0 = s1;
                } while (kParts && s0 < t.kb1);
            }
            // every MMA issued above completes before the CTA leaves
            mma_commit_elect<2>(smem_u32(&ctl->mma_done), 1);
            if (lane == 0) {
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(smem_u32(&ctl->mma_done), 0) && global_timer_ns() - t0 < a.timeout_ns) {}
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------ odd CTA: reports its half of B
            if (kKeepB && first < a.items && tile_wait_warp(a, ctl, &ctl->b_full[0], 0) && lane == 0)
                mbar_arrive_remote(map_shared_rank(smem_u32(&ctl->b_full[0]), 0));
            for (int64_t it = first; it < a.items && ok && !kKeepB; it += step) {
                const TileItem t = tile_item<kTN>(a, it, rank);
                for (int32_t kb = t.kb0; kb < t.kb1; ++kb) {
                    if (!tile_wait_warp(a, ctl, &ctl->b_full[ring], ring_phase)) { ok = false; break; }
                    if (lane == 0) mbar_arrive_remote(map_shared_rank(smem_u32(&ctl->ready[ring]), 0));
                    if (++ring == kTileRing) { ring = 0; ring_phase ^= 1u; }
                }
            }
        }
    }
    } else if (warp < kTileEpiWarp0) {
        regs_release<tile_regs_widen(sizeof(T) == 2)>();
        // ------------------------------------------------------------ widening
        const int wg = (warp - kWidenWarp0) >> 2, q = warp & 3;
        const int row = q * 32 + lane;
        const uint32_t a_lane = tmem + (static_cast<uint32_t>(q * 32) << 16) + kTileACol;
        int32_t stage = 0, ring = 0;
        uint32_t phase = 0, ring_phase = 0;
        int turn = 0;
        bool ok = true;
        for (int64_t it = first; it < a.items && ok; it += step) {
            const TileItem t = tile_item<kTN>(a, it, rank);
            for (int32_t kb = t.kb0; kb < t.kb1; ++kb) {
                if (turn == wg) {
                    if (!tile_wait_warp(a, ctl, &ctl->full8[stage], phase)) { ok = false; break; }
                    const uint8_t* src = s8 + stage * C::kA8 + row * kTileK;
                    uint4 v[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[c] = *reinterpret_cast<const uint4*>(src + ((c ^ (row & 7)) << 4));
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&ctl->empty8[stage]));
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t h[32];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t e[8];
                            widen16(v[half * 4 + c], e);
#pragma unroll
                            for (int i = 0; i < 8; ++i) h[c * 8 + i] = e[i];
                        }
                        if (half == 0) {  // the MMAs that read the slot's last block are done
                            if (!tile_wait_warp(a, ctl, &ctl->freed[ring], ring_phase ^ 1u)) { ok = false; break; }
                            tc_fence_after();
                        }
                        tmem_st32(a_lane + static_cast<uint32_t>(ring * 64 + half * 32), h);
                    }
                    if (!ok) break;
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(map_shared_rank(smem_u32(&ctl->ready[ring]), 0));
                }
                turn ^= 1;
                if (++stage == C::kStages8) { stage = 0; phase ^= 1u; }
                if (++ring == kTileRing) { ring = 0; ring_phase ^= 1u; }
            }
        }
    } else {
        regs_claim<tile_regs_epi(sizeof(T) == 2)>();
        // ------------------------------------------------------------ epilogue
        // A warp owns 32 rows of A and half of the tile's columns; in the
        // accumulator a lane holds a row. 16-bit outputs are scaled, rounded and
        // held in registers until the accumulator has been read and handed
        // back, so that only this stands between a tile's MMAs and the next
        // one's. The scales along B wait in shared memory, where a read serves
        // the whole warp. Rows of 16-bit outputs then pass through shared memory
        // to TMA stores (139270 x 1864 x 64 bf16 209 -> 148 us from 16-byte
        // stores of the warps, most of it their instructions; 135 now). Swapped, lanes are
        // consecutive channels and store straight to out. 32-bit outputs, and
        // the integer sums of slices, are stored 32 columns at a time as they
        // are read, through shared memory so that stores are whole 128-byte runs.
        const int q = warp & 3, half = (warp - kTileEpiWarp0) >> 2;
        constexpr int kCols = kTN / 2, kChunks = kCols / 32;  // columns per warp
        constexpr bool kHold = sizeof(T) == 2, kTma = kHold && kRows16 && !kSwap;
        uint8_t* stage = s_out + (warp - kTileEpiWarp0) * kTileStage;
        float* tab = reinterpret_cast<float*>(stage);  // kHold: scales of the kCols columns, then biases
        const int64_t ld = kSums ? a.l.N : a.l.ld_out;
        int32_t buf = 0;
        uint32_t buf_phase = 0;
        // this lane's row of A, and its column of each 32 along B. Loaded an item
        // ahead where registers are left for it (us ahead / not: 603311 x 64 x 64 bf16 36 / 44,
        // 999 x 1537 x 1111 f32 11.4 / 12.0, 525402 x 960 x 64 f32 418 / 425, but 139270 x 1864 x
        // 176 f32 262 / 248), not beside the held outputs of wide tiles (202805 x 576 x 64 bf16
        // 80 / 73, 2048 x 4096 x 1024 bf16 18.5 / 18.1)
        constexpr bool kAhead = !kHold || kTN == 64;
        float next_sa = 0.f, next_bias_a = 0.f, next_sb[kChunks], next_bias[kSwap ? 1 : kChunks];
        auto load_scales = [&](const TileItem& t) {
            if constexpr (kSums) return;
            const int64_t ra = t.a0 + q * 32 + lane;
            const bool in = ra < a.rows_a;
            next_sa = in ? __ldg((kSwap ? a.l.w_scale : a.l.x_scale) + ra) : 0.f;
            if constexpr (kSwap) next_bias_a = a.l.bias && in ? __ldg(a.l.bias + ra) : 0.f;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int64_t i = t.b0 + half * kCols + c * 32 + lane;
                next_sb[c] = i < a.rows_b ? __ldg((kSwap ? a.l.x_scale : a.l.w_scale) + i) : 0.f;
                if constexpr (!kSwap) next_bias[c] = a.l.bias && i < a.rows_b ? __ldg(a.l.bias + i) : 0.f;
            }
        };
        if constexpr (kAhead) load_scales(tile_item<kTN>(a, first, rank));
        for (int64_t it = first; it < a.items; it += step) {
            const TileItem t = tile_item<kTN>(a, it, rank);
            if constexpr (!kAhead) load_scales(t);
            const int64_t ra0 = t.a0 + q * 32, rb0 = t.b0 + half * kCols;
            T* out = static_cast<T*>(a.l.out);
            if constexpr (kSums) out = a.partial + static_cast<int64_t>(t.slice) * a.l.M * a.l.N;
            const int row_n = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(32), a.rows_a - ra0)));
            const bool in_a = lane < row_n;
            const float sa = next_sa, bias_a = next_bias_a;
            const float2 sa2 = make_float2(sa, sa);
            float sb[kHold ? 1 : kChunks], bias[kHold || kSwap ? 1 : kChunks];
            if constexpr (kTma) {  // the table is written where the last tile's stores read
                if (lane == 0) bulk_wait_read();
                __syncwarp();
            }
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if constexpr (kHold) {
                    tab[c * 32 + lane] = next_sb[c];
                    if constexpr (!kSwap) tab[kCols + c * 32 + lane] = next_bias[c];
                } else {
                    sb[c] = next_sb[c];
                    if constexpr (!kSwap) bias[c] = next_bias[c];
                }
            }
            __syncwarp();
            if (kAhead && it + step < a.items) load_scales(tile_item<kTN>(a, it + step, rank));
            const uint32_t src0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * kCols);
            int32_t sum[kParts ? kCols : 1];
            if constexpr (kParts) {  // two floats as such (conversions are slow): see parts_needed
                bool ok = true;
                const bool as_float = !kSums && t.kb1 - t.kb0 <= 2 * a.kb_part;
                for (int32_t s0 = t.kb0; s0 < t.kb1; s0 += a.kb_part) {
                    if (!(ok = tile_wait_warp(a, ctl, &ctl->acc_full[buf], buf_phase))) break;
                    tc_fence_after();
                    float v[2][16];
                    const uint32_t from = src0 + static_cast<uint32_t>(buf * kTN);
                    tmem_ld16(from, v[0]);
#pragma unroll
                    for (int c = 0; c < kCols; c += 16) {
                        float (&u)[16] = v[(c / 16) & 1];
                        tmem_wait_ld16(u);
                        if (c + 16 < kCols) {
                            tmem_ld16(from + c + 16, v[(c / 16 + 1) & 1]);
                        } else {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_remote(map_shared_rank(smem_u32(&ctl->acc_empty[buf]), 0));
                        }
                        if (as_float) {
                            const bool start = s0 == t.kb0;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                sum[c + i] = __float_as_int(start ? u[i] : __int_as_float(sum[c + i]) + u[i]);
                        } else {
                            const int32_t keep = s0 == t.kb0 ? 0 : -1;
#pragma unroll
                            for (int i = 0; i < 16; ++i) sum[c + i] = (sum[c + i] & keep) + __float2int_rn(u[i]);
                        }
                    }
                    if (s0 + a.kb_part < t.kb1 && ++buf == C::kAcc) { buf = 0; buf_phase ^= 1u; }
                }
                if (!ok) break;
                if (!kSums && !as_float) {
#pragma unroll
                    for (int i = 0; i < kCols; ++i) sum[i] = __float_as_int(__int2float_rn(sum[i]));
                }
            } else {
                if (!tile_wait_warp(a, ctl, &ctl->acc_full[buf], buf_phase)) break;
                tc_fence_after();
            }
            const uint32_t src = src0 + static_cast<uint32_t>(buf * kTN);
            uint32_t held[kHold ? kChunks : 1][16];
            if constexpr (kHold) {
                // one part is in flight while another is worked on (2048 x 4096 x 1024 bf16 19.6 -> 18.7 us)
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
                        if (lane == 0) mbar_arrive_remote(map_shared_rank(smem_u32(&ctl->acc_empty[buf]), 0));
                    }
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 s4 = *reinterpret_cast<const float4*>(tab + c * 16 + i);
                        const float4 b4 = kSwap ? make_float4(bias_a, bias_a, bias_a, bias_a)
                                                : *reinterpret_cast<const float4*>(tab + kCols + c * 16 + i);
                        const float* u = v[c & 1] + i;
                        const float2 lo = fma2(mul2(make_float2(u[0], u[1]), sa2), make_float2(s4.x, s4.y), make_float2(b4.x, b4.y));
                        const float2 hi = fma2(mul2(make_float2(u[2], u[3]), sa2), make_float2(s4.z, s4.w), make_float2(b4.z, b4.w));
                        held[c / 2][(c & 1) * 8 + i / 2] = pack2<T>(lo.x, lo.y);
                        held[c / 2][(c & 1) * 8 + i / 2 + 1] = pack2<T>(hi.x, hi.y);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < kChunks && !kHold; ++c) {
                const int64_t rb = rb0 + c * 32;
                float v[32];  // kSums: integers as their bits
                if constexpr (kParts) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __int_as_float(sum[c * 32 + i]);
                } else {
                    tmem_ld32(src + c * 32, v);
                    tmem_wait_ld();
                    if (c + 1 == kChunks) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(map_shared_rank(smem_u32(&ctl->acc_empty[buf]), 0));
                    }
                }
                if (row_n == 0 || rb >= a.rows_b) continue;
                if constexpr (kSums && !kParts) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __int_as_float(__float2int_rn(v[i]));
                }
                if constexpr (kSwap) {
                    const int n = static_cast<int>(min(static_cast<int64_t>(32), a.rows_b - rb));
                    T* p = out + rb * ld + ra0 + lane;
#pragma unroll
                    for (int i = 0; i < 32; ++i, p += ld) {
                        float y = v[i];
                        if constexpr (!kSums) y = __fmaf_rn(y * __shfl_sync(0xffffffffu, sb[c], i), sa, bias_a);
                        if (i < n && in_a) *p = from_f32<T>(y);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4*>(stage + staged(lane, i)) =
                            kSums ? make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3])
                                  : make_float4(v[4 * i] * sa, v[4 * i + 1] * sa, v[4 * i + 2] * sa, v[4 * i + 3] * sa);
                    __syncwarp();
                    if constexpr (kRows16) {
                        float ws[4] = {}, bs[4] = {};  // this lane's four channels
                        if constexpr (!kSums && !kHold) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                ws[j] = __shfl_sync(0xffffffffu, sb[c], 4 * (lane & 7) + j);
                                bs[j] = __shfl_sync(0xffffffffu, bias[c], 4 * (lane & 7) + j);
                            }
                        }
                        const int64_t n0 = rb + 4 * (lane & 7);
                        const int n = static_cast<int>(min(static_cast<int64_t>(4), a.rows_b - n0));
                        int64_t at = (ra0 + (lane >> 3)) * ld + n0;
#pragma unroll
                        for (int i = 0; i < 8; ++i, at += 4 * ld) {
                            const float4 y = *reinterpret_cast<const float4*>(stage + staged(4 * i + (lane >> 3), lane & 7));
                            if (4 * i + (lane >> 3) >= row_n) continue;
                            if constexpr (kSums) {
                                store4(out + at, n, y.x, y.y, y.z, y.w);
                            } else if constexpr (!kHold) {
                                store4(out + at, n, __fmaf_rn(y.x, ws[0], bs[0]), __fmaf_rn(y.y, ws[1], bs[1]),
                                       __fmaf_rn(y.z, ws[2], bs[2]), __fmaf_rn(y.w, ws[3], bs[3]));
                            }
                        }
                    } else {  // rows off their 16-byte boundaries: a row at a time, a lane per column
                        const bool in_b = rb + lane < a.rows_b;
                        const uint8_t* from = stage + (lane & 3) * 4;
                        int64_t at = ra0 * ld + rb + lane;
#pragma unroll 8
                        for (int r = 0; r < row_n; ++r, at += ld) {
                            float y = *reinterpret_cast<const float*>(from + staged(r, lane >> 2));
                            if constexpr (!kSums && !kHold) y = __fmaf_rn(y, sb[c], bias[c]);
                            if (in_b) out[at] = from_f32<T>(y);
                        }
                    }
                    __syncwarp();
                }
            }
            if constexpr (kHold) {
                if (row_n > 0) {
                    __syncwarp();  // the table is done with
                    if constexpr (kSwap) {
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {
                            const int64_t rb = rb0 + c * 32;
                            const int n = static_cast<int>(min(static_cast<int64_t>(32), a.rows_b - rb));
                            T* p = out + rb * ld + ra0 + lane;
#pragma unroll
                            for (int i = 0; i < 32; ++i, p += ld)
                                if (i < n && in_a) *p = half_of<T>(held[c][i / 2], i & 1);
                        }
                    } else if constexpr (kTma) {
                        constexpr int kJoin = kChunks < 2 ? 1 : 2;  // chunks that are staged and stored together
#pragma unroll
                        for (int c = 0; c < kChunks; c += kJoin) {
                            const int64_t n0 = rb0 + c * 32;
                            if (n0 >= a.rows_b) break;
                            if (c > 0) {
                                if (lane == 0) bulk_wait_read();
                                __syncwarp();
                            }
#pragma unroll
                            for (int j = 0; j < 4 * kJoin; ++j)
                                *reinterpret_cast<uint4*>(stage + boxed<kJoin>(lane, j)) =
                                    make_uint4(held[c + j / 4][(j % 4) * 4], held[c + j / 4][(j % 4) * 4 + 1],
                                               held[c + j / 4][(j % 4) * 4 + 2], held[c + j / 4][(j % 4) * 4 + 3]);
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) tma_store_2d(&tm_out, smem_u32(stage), static_cast<int32_t>(n0), static_cast<int32_t>(ra0));
                        }
                    } else {
                        // Rows off their 16-byte boundaries. Every lane turns its row by the
                        // phase of its address, so that staged pieces are pieces of out; the
                        // first one holds the row's first elements and, wrapped around, its last
                        // ones, which go out one by one. (139270 x 1861 x 176 bf16: 712 us with
                        // single elements throughout, 427 joining pieces at the store, 311 so; 244 now.)
                        constexpr int kJoin = kChunks < 2 ? 1 : 2;         // chunks whose rows are staged together
                        constexpr int kRun = 32 * kJoin, kPieces = kRun / 8, kRows = 32 / kPieces;
                        auto phase_of = [](const T* p) { return static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 1) & 7; };
                        const int k = lane % kPieces, r0 = lane / kPieces;
#pragma unroll
                        for (int c = 0; c < kChunks; c += kJoin) {
                            const int64_t n0 = rb0 + c * 32;
                            if (n0 >= a.rows_b) break;
                            const int left = static_cast<int>(min(static_cast<int64_t>(kRun), a.rows_b - n0));
                            T* const out0 = out + ra0 * ld + n0;
                            const int turn = phase_of(out0 + lane * ld);
                            uint32_t v[kRun / 2], u[kRun / 2];
#pragma unroll
                            for (int i = 0; i < kRun / 2; ++i) v[i] = held[c + i / 16][i % 16];
#pragma unroll
                            for (int i = 0; i < kRun / 2; ++i)
                                u[i] = __funnelshift_l(v[(i + kRun / 2 - 1) % (kRun / 2)], v[i], (turn & 1) * 16);
#pragma unroll
                            for (int i = 0; i < kRun / 2; ++i) v[i] = turn & 2 ? u[(i + kRun / 2 - 1) % (kRun / 2)] : u[i];
#pragma unroll
                            for (int i = 0; i < kRun / 2; ++i) u[i] = turn & 4 ? v[(i + kRun / 2 - 2) % (kRun / 2)] : v[i];
#pragma unroll
                            for (int j = 0; j < kPieces; ++j)
                                *reinterpret_cast<uint4*>(stage + staged(lane, j)) =
                                    make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
                            __syncwarp();
                            T* p = out0 + r0 * ld;
#pragma unroll
                            for (int i = 0; i < kPieces; ++i, p += kRows * ld) {
                                const int r = i * kRows + r0, ph = phase_of(p);
                                const uint4 y = *reinterpret_cast<const uint4*>(stage + staged(r, k));
                                if (r < row_n && (k > 0 || ph == 0) && 8 * k - ph + 8 <= left)
                                    *reinterpret_cast<uint4*>(p + 8 * k - ph) = y;
                            }
                            p = out0 + (lane >> 3) * ld;
                            const int e = lane & 7;
#pragma unroll
                            for (int i = 0; i < 8; ++i, p += 4 * ld) {
                                const int r = i * 4 + (lane >> 3), ph = phase_of(p), col = e < ph ? kRun - ph + e : e - ph;
                                const T y = *reinterpret_cast<const T*>(stage + staged(r, 0) + e * 2);
                                if (r < row_n && ph != 0 && col < left) p[col] = y;
                            }
                            if (left < kRun) {  // the last columns: the end of a row is not yet in its first piece
                                p = out0 + (lane >> 3) * ld;
#pragma unroll
                                for (int i = 0; i < 8; ++i, p += 4 * ld) {
                                    const int r = i * 4 + (lane >> 3), ph = phase_of(p), end = (left + ph) >> 3;
                                    const T y = *reinterpret_cast<const T*>(stage + staged(r, end % kPieces) + e * 2);
                                    if (r < row_n && e < ((left + ph) & 7) && end < kPieces && (end > 0 || ph == 0))
                                        p[8 * end - ph + e] = y;
                                }
                            }
                            __syncwarp();
                        }
                    }
                }
            }
            if (++buf == C::kAcc) { buf = 0; buf_phase ^= 1u; }
        }
        if (kTma && lane == 0) bulk_wait();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // no CTA leaves while its pair may still touch it
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc<2>(tmem, 512);
    }
}

// Adds the slices' integer sums, scales, adds the bias and rounds once.
template <typename T>
__global__ void __launch_bounds__(256) linear_join_kernel(const LinearArgs l, const int32_t* __restrict__ partial,
                                                          int32_t slices) {
    const int64_t n_out = static_cast<int64_t>(l.M) * l.N;
    wait_for_previous();
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n_out;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t m = i / l.N, n = i - m * l.N;
        int32_t sum = 0;
        for (int32_t s = 0; s < slices; ++s) sum += partial[s * n_out + i];
        float v = static_cast<float>(sum) * l.x_scale[m] * l.w_scale[n];
        if (l.bias) v += l.bias[n];
        static_cast<T*>(l.out)[m * l.ld_out + n] = from_f32<T>(v);
    }
}

}  // namespace maxsim
