// Rows of 4-bit floating-point values (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and
// their negatives) with a scale for every block of 16 or 32 of them: the
// quantisation of rows and its reverse.
//
// Layout, as the block-scaled MMAs read it: a row's codes are whole 16-byte
// pieces (32 values, the lower index in the low half of a byte, zeros behind
// the row's end); the scales of four consecutive blocks of a row are one
// 32-bit word, and the words of 128 rows are a tile of 512 bytes in which row
// r's stands at byte (r % 32) * 16 + (r / 32) * 4, tiles of the same rows one
// after another. Rows of a tile and blocks of a word that do not exist have
// the scale byte 0.
#pragma once

#include <cstdint>
#include <type_traits>

#include "head_kernels.cuh"
#include "tile_store.cuh"

namespace maxsim {

// ---------------------------------------------------------------- conversions

// Eight floats to four bytes of codes (the first in the low half of the first byte), nearest, ties to even, 6 at most.
__device__ __forceinline__ uint32_t to_e2m1x8(const float* v) {
    uint32_t d;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(d) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

// Eight codes to four pairs of binary16 (exact).
__device__ __forceinline__ void from_e2m1x8(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(codes));
}

// The E4M3 value nearest to v >= 0 (ties to even, 448 at most), and what a byte stands for.
__device__ __forceinline__ uint32_t to_e4m3(float v) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.f), "f"(v));
    return d & 0xffu;
}
__device__ __forceinline__ float from_e4m3(uint32_t byte) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffffu)));
}
// What an E8M0 byte stands for: 2^(byte - 127), 255 is NaN.
__device__ __forceinline__ float from_e8m0(uint32_t byte) {
    if (byte == 255u) return __uint_as_float(0x7fffffffu);
    return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}
template <int kBlock>
__device__ __forceinline__ float block_scale_value(uint32_t byte) {
    return kBlock == 16 ? from_e4m3(byte) : from_e8m0(byte);
}

// Byte of the scale word of row r's blocks 4 j .. 4 j + 3, of `words` words a row.
__host__ __device__ __forceinline__ int64_t scale_word_at(int64_t r, int64_t j, int64_t words) {
    return ((r >> 7) * words + j) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// 32 bytes on a 32-byte boundary in one load or store.
__device__ __forceinline__ void load32(const void* p, uint32_t (&v)[8]) {
    asm("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]) : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "l"(p)
                 : "memory");
}

// ---------------------------------------------------------------- 16 elements of a row

template <typename T>
struct Sixteen {
    static constexpr int kWords = static_cast<int>(sizeof(T)) * 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const T* p) {  // p on a 32-byte boundary
#pragma unroll
        for (int i = 0; i < kWords; i += 8) load32(reinterpret_cast<const uint32_t*>(p) + i, reinterpret_cast<uint32_t(&)[8]>(w[i]));
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < kWords; i += 8)
            store32(reinterpret_cast<uint32_t*>(p) + i, reinterpret_cast<const uint32_t(&)[8]>(w[i]));
    }
    __device__ __forceinline__ void set(int i, uint32_t bits) {  // into cleared words
        if constexpr (sizeof(T) == 4) w[i] = bits;
        else w[i >> 1] |= bits << ((i & 1) * 16);
    }
    static __device__ __forceinline__ uint32_t bits_of(const T* p) {
        if constexpr (sizeof(T) == 4) return *reinterpret_cast<const uint32_t*>(p);
        else return *reinterpret_cast<const unsigned short*>(p);
    }
    // from any element's address: the aligned 16-byte pieces that hold them, shifted into place
    __device__ __forceinline__ void load_any(const T* p) {
        constexpr int kPieces = kWords / 4 + 1;
        const uintptr_t from = reinterpret_cast<uintptr_t>(p);
        const uint4* q = reinterpret_cast<const uint4*>(from & ~uintptr_t(15));
        const uint32_t by = static_cast<uint32_t>(from) & 15u;
        uint32_t v[4 * kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint4 u = i + 1 < kPieces || by ? __ldg(q + i) : make_uint4(0, 0, 0, 0);
            v[4 * i] = u.x; v[4 * i + 1] = u.y; v[4 * i + 2] = u.z; v[4 * i + 3] = u.w;
        }
        if (by & 8u) {
#pragma unroll
            for (int i = 0; i + 2 < 4 * kPieces; ++i) v[i] = v[i + 2];
        }
        if (by & 4u) {
#pragma unroll
            for (int i = 0; i + 1 < 4 * kPieces; ++i) v[i] = v[i + 1];
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = sizeof(T) == 4 ? v[i] : __funnelshift_r(v[i], v[i + 1], (by & 2u) * 8);
    }
    // the first n >= 1 elements from p, one by one (all loads before their first use)
    __device__ __forceinline__ void load_some(const T* p, int n) {
        uint32_t e[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) e[i] = bits_of(p + min(i, n - 1));
        clear();
#pragma unroll
        for (int i = 0; i < 16; ++i) set(i, i < n ? e[i] : 0u);
    }
    // zeros from element n on
    __device__ __forceinline__ void keep(int n) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 4) w[i] = i < n ? w[i] : 0u;
            else w[i] = 2 * i + 1 < n ? w[i] : 2 * i < n ? w[i] & 0xffffu : 0u;
        }
    }
    // To any element's address, by lanes whose neighbours hold the elements behind
    // theirs (at most kLanes of them together; every lane of the warp calls it). `left`:
    // elements of the row from p on (<= 0: none). A lane stores the aligned 16-byte
    // pieces that begin among its elements, the last of them with its neighbour's
    // first elements; the elements around all of them go one by one.
    template <int kLanes>
    __device__ __forceinline__ void store_any(T* p, int left) const {
        constexpr int kVec = 16 / static_cast<int>(sizeof(T)), kMore = 4;  // words of the neighbour
        const int l = static_cast<int>(threadIdx.x) % kLanes;
        uint32_t u[kWords + kMore];
#pragma unroll
        for (int i = 0; i < kWords; ++i) u[i] = w[i];
#pragma unroll
        for (int i = 0; i < kMore; ++i) u[kWords + i] = __shfl_down_sync(0xffffffffu, w[i], 1);
        const int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / static_cast<int>(sizeof(T));
        const int own = left < 16 ? left : l + 1 == kLanes ? 16 : left;  // elements from p on that this lane may store
        const int by = head * static_cast<int>(sizeof(T));  // bytes
        if (by & 8) {
#pragma unroll
            for (int i = 0; i + 2 < kWords + kMore; ++i) u[i] = u[i + 2];
        }
        if (by & 4) {
#pragma unroll
            for (int i = 0; i + 1 < kWords + kMore; ++i) u[i] = u[i + 1];
        }
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i + 1 < kWords + kMore; ++i) u[i] = __funnelshift_r(u[i], u[i + 1], (by & 2) * 8);
        }
        int done = head;
#pragma unroll
        for (int k = 0; k < 16 / kVec; ++k) {
            if (head + k * kVec + kVec <= own) {
                *reinterpret_cast<uint4*>(p + head + k * kVec) = make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
                done = head + k * kVec + kVec;
            }
        }
        // in front: the first lane's, or where the lane before has no piece to take them; behind: what no piece took
        const bool front = l == 0 || left < head;
        if (front || done < min(left, 16)) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < left && ((front && i < head) || i >= done)) p[i] = element(i);
        }
    }
    __device__ __forceinline__ T element(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return half_of<T>(w[i >> 1], i & 1);
    }
    // elements 2 i and 2 i + 1
    __device__ __forceinline__ float2 pair(int i) const {
        if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return unpack2<T>(w[i]);
    }
    // max |.| as the bits of a float (infinities and NaN on top)
    __device__ __forceinline__ uint32_t largest() const {
        uint32_t m = 0;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7fffffffu);
            return m;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max_u16x2(m, w[i] & 0x7fff7fffu);
            m = max(m >> 16, m & 0xffffu);
            if constexpr (std::is_same_v<T, __half>) return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
            else return m << 16;
        }
    }
};

// ---------------------------------------------------------------- quantisation

struct Fp4QuantizeArgs {
    const void* x;
    uint8_t* q;
    uint8_t* block_scale;
    float* scale;  // block 16
    int64_t rows, ld_x, ld_q;
    int32_t cols;
    int32_t chunks;  // of 16 values that q has: 2 * ceil(cols / 32)
    int32_t words;   // scale words of a row
};

constexpr uint32_t kInfBits = 0x7f800000u;

// The row's scale of block 16: the smallest power of two s >= 2^-126 with
// max |x| <= 448 * 6 * s (448 * 6 = 1.3125 * 2^11), as its exponent.
__device__ __forceinline__ int row_exponent(uint32_t largest) {
    const int e = static_cast<int>(largest >> 23) - 127 - 11 + ((largest & 0x7fffffu) > 0x280000u ? 1 : 0);
    return max(e, -126);
}

// 1 / b to twice fp32's digits: hi + lo with hi <= 1 / b, so that lo >= 0.
__device__ __forceinline__ float2 reciprocal(float b) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b));
    float e = __fmaf_rn(-r, b, 1.f);
    if (e < 0.f) {
        r = __uint_as_float(__float_as_uint(r) - 2u);
        e = __fmaf_rn(-r, b, 1.f);
    }
    return make_float2(r, e * r);
}

// Codes of 16 elements, and their block's scale byte.
//  block 16: with y = x / s (exact, s a power of two), b = max(e4m3(max |y| / 6), 2^-9), code = e2m1(y / b).
//  A quotient within a rounding of a code's border would change the code. So it
//  is rounded once: y * hi + y * lo with 1 / b = hi + lo to 2^-46 of itself. A
//  quotient rounded so never sits on a border that the exact one is off: borders
//  times b have at most seven bits, and a 24-bit y next to one is further away
//  than half a step of the quotient, by 6 % of it at least. The same holds of
//  max |y| / 6 and the borders of E4M3. (lo >= 0 keeps the sign of -0.)
//  block 32: b = 2^(floor(log2 max |x|) - 2), at least 2^-127; x / b is exact.
template <typename T, int kBlock>
__device__ __forceinline__ uint2 code16(const Sixteen<T>& v, uint32_t block_max, float inv_row, uint32_t* byte) {
    float y[16];
    if constexpr (kBlock == 16) {
        constexpr float kSixth = 0x1.555554p-3f, kSixthLo = 0x1.555556p-27f;  // 1 / 6 cut to 24 bits, and what is left of it
        const float most = __uint_as_float(block_max) * inv_row;
        const uint32_t c = max(to_e4m3(__fmaf_rn(most, kSixth, most * kSixthLo)), 1u);
        *byte = c;
        const float2 r = reciprocal(from_e4m3(c)), hi = make_float2(r.x, r.x), lo = make_float2(r.y, r.y), inv = make_float2(inv_row, inv_row);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 x = mul2(v.pair(i), inv), q = fma2(x, hi, mul2(x, lo));
            y[2 * i] = q.x;
            y[2 * i + 1] = q.y;
        }
    } else {
        const uint32_t field = block_max >> 23, c = field > 2 ? field - 2 : 0;
        *byte = c;
        const float inv = __uint_as_float((254u - c) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 q = mul2(v.pair(i), make_float2(inv, inv));
            y[2 * i] = q.x;
            y[2 * i + 1] = q.y;
        }
    }
    return make_uint2(to_e2m1x8(y), to_e2m1x8(y + 8));
}

// A chunk's codes to q (NULL: it has none), and its share of the row's scale word;
// the word is gathered from the lanes of the row's neighbouring chunks (lanes of
// a group hold consecutive chunks) and stored by the first of them (word not NULL).
template <typename T, int kBlock, int kGroup>
__device__ __forceinline__ void store16(const Sixteen<T>& v, int32_t chunk, bool finite, float inv_row, uint8_t* q, bool has_scale, uint32_t* word) {
    uint32_t m = v.largest(), byte;
    if constexpr (kBlock == 32) {
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        finite = m < kInfBits;
    }
    uint2 codes = code16<T, kBlock>(v, finite ? m : 0u, inv_row, &byte);
    if (!finite) {  // block 16: the row's scale is NaN
        codes = make_uint2(0, 0);
        if (kBlock == 32) byte = 255u;
    }
    if (q) *reinterpret_cast<uint2*>(q) = codes;
    constexpr int kPer = kBlock == 16 ? 4 : 8;  // chunks of a word
    uint32_t w = has_scale ? byte << (kBlock == 16 ? (chunk & 3) * 8 : ((chunk >> 1) & 3) * 8) : 0u;
#pragma unroll
    for (int o = 1; o < kPer && o < kGroup; o <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, o);
    if (word) *word = w;
}

// Whether a chunk has a scale byte to write, and whether it writes its scale word.
template <int kBlock>
__device__ __forceinline__ bool chunk_has_scale(const Fp4QuantizeArgs& a, int32_t chunk) {
    return static_cast<int64_t>(chunk) * 16 < a.cols && (kBlock == 16 || (chunk & 1) == 0);
}
template <int kBlock>
__device__ __forceinline__ bool chunk_has_word(const Fp4QuantizeArgs& a, int32_t chunk) {
    constexpr int kPer = kBlock == 16 ? 4 : 8;
    return chunk % kPer == 0 && chunk / kPer < a.words;
}

// Loads `n` <= 16 elements of a chunk from p (n <= 0: none). kWide: p is on a
// 32-byte boundary. A chunk that reaches over its row's end is read as a whole
// where the operand goes on, and cut.
template <typename T, bool kWide>
__device__ __forceinline__ void load16(Sixteen<T>& v, const T* p, int32_t n, const T* base, const T* end) {
    if (n <= 0) {
        v.clear();
        return;
    }
    if constexpr (kWide) {
        if (n == 16) {
            v.load(p);
            return;
        }
        if (p + 16 <= end) v.load(p);
        else v.load_some(p, n);
    } else {
        const uintptr_t first = reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15), last = (reinterpret_cast<uintptr_t>(p + 16) + 15) & ~uintptr_t(15);
        if (first >= reinterpret_cast<uintptr_t>(base) && last <= reinterpret_cast<uintptr_t>(end)) v.load_any(p);
        else v.load_some(p, n);
    }
    if (n < 16) v.keep(n);
}

__host__ __device__ constexpr int fp4_threads(int group) { return group < 256 ? 256 : group; }
// Rows whose loads a group has in flight together: two where a thread has one chunk
// of a row (5000000 x 128 f16 285 -> 239 us), one where registers are short (262144 x
// 1023 bf16 off its boundaries 141 us, with two 212).
__host__ __device__ constexpr int fp4_flight(int group, int chunks, bool wide) { return group <= 32 && chunks == 1 && wide ? 2 : 1; }

// A row's 16-element chunks lie in the registers of a group of kGroup threads,
// kChunks each, between the row's maximum (block 16 needs it before the first
// code) and the codes: x is read once. The rows of all blocks together are a
// multiple of 128, so a thread's rows have the same place in their scale tiles and
// all its addresses go on by constant steps. Bound by HBM for f32 and for block
// 32, by the instructions for 16-bit rows with block 16 (5000000 x 128 f16, 239 us
// at HBM's rate: block 32 238 us, block 16 313).
template <typename T, int kBlock, bool kWide, int kGroup, int kChunks>
__global__ void __launch_bounds__(fp4_threads(kGroup)) fp4_quantize_kernel(const Fp4QuantizeArgs a) {
    constexpr int kThreads = fp4_threads(kGroup), kRows = kThreads / kGroup, kFlight = fp4_flight(kGroup, kChunks, kWide);
    __shared__ uint32_t slot[2][kThreads / 32];
    const int t = threadIdx.x % kGroup;
    const uint32_t rows = static_cast<uint32_t>(a.rows), padded = (rows + 127u) & ~127u, step = gridDim.x * kRows;
    const T* base = static_cast<const T*>(a.x);
    const T* end = base + (a.rows - 1) * a.ld_x + a.cols;
    int32_t n[kChunks];
    bool has_code[kChunks], has_scale[kChunks], has_word[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int32_t chunk = c * kGroup + t;
        n[c] = static_cast<int32_t>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(16), a.cols - static_cast<int64_t>(chunk) * 16)));
        has_code[c] = chunk < a.chunks;
        has_scale[c] = chunk_has_scale<kBlock>(a, chunk);
        has_word[c] = chunk_has_word<kBlock>(a, chunk);
    }
    const uint32_t row0 = blockIdx.x * kRows + threadIdx.x / kGroup;
    const T* x = base + static_cast<int64_t>(row0) * a.ld_x + t * 16;
    uint8_t* q = a.q + static_cast<int64_t>(row0) * a.ld_q + t * 8;
    constexpr int kPer = kBlock == 16 ? 4 : 8;
    uint8_t* word = a.block_scale + scale_word_at(row0, t / kPer, a.words);
    const int64_t x_step = static_cast<int64_t>(step) * a.ld_x, q_step = static_cast<int64_t>(step) * a.ld_q,
                  word_step = static_cast<int64_t>(step >> 7) * a.words * 512;
    int turn = 0;
    // a block's rows are all of a tile's or none, so its threads stay together
    for (uint32_t r0 = blockIdx.x * kRows; r0 < padded; r0 += kFlight * step) {
        Sixteen<T> v[kFlight][kChunks];
#pragma unroll
        for (int f = 0; f < kFlight; ++f)
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                load16<T, kWide>(v[f][c], x + f * x_step + c * kGroup * 16, row0 - blockIdx.x * kRows + r0 + f * step < rows ? n[c] : 0, base, end);
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const uint32_t first = r0 + f * step;
            if (f > 0 && first >= padded) break;
            const uint32_t row = first + threadIdx.x / kGroup;
            const bool row_in = row < rows;
            float inv_row = 1.f;
            bool finite = true;
            if constexpr (kBlock == 16) {
                uint32_t m = 0;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) m = max(m, v[f][c].largest());
                if constexpr (kGroup <= 32) {
                    m = group_max<kGroup>(m, nullptr);
                } else {  // groups of a block's warps
                    m = __reduce_max_sync(0xffffffffu, m);
                    if ((threadIdx.x & 31) == 0) slot[turn][threadIdx.x >> 5] = m;
                    __syncthreads();
                    const int w0 = static_cast<int>(threadIdx.x) / kGroup * (kGroup / 32);
                    m = __reduce_max_sync(0xffffffffu, slot[turn][w0 + (threadIdx.x & 31) % (kGroup / 32)]);
                    turn ^= 1;
                }
                finite = m < kInfBits;
                const int e = finite ? row_exponent(m) : 0;
                inv_row = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                if (row_in && t == 0) a.scale[row] = finite ? __uint_as_float(static_cast<uint32_t>(127 + e) << 23) : __uint_as_float(0x7fffffffu);
            }
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                store16<T, kBlock, kGroup>(v[f][c], c * kGroup + t, finite, inv_row, row_in && has_code[c] ? q + f * q_step + c * kGroup * 8 : nullptr,
                                           row_in && has_scale[c],
                                           has_word[c] ? reinterpret_cast<uint32_t*>(word + f * word_step + c * (kGroup / kPer) * 512) : nullptr);
        }
        x += kFlight * x_step;
        q += kFlight * q_step;
        word += kFlight * word_step;
    }
}

// Rows that no group holds: a block per row, read twice with block 16.
template <typename T, int kBlock, bool kWide>
__global__ void __launch_bounds__(512) fp4_quantize_long_kernel(const Fp4QuantizeArgs a) {
    __shared__ uint32_t slot[2][16];
    const int64_t padded = (a.rows + 127) / 128 * 128;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < padded; row += gridDim.x, turn ^= 1) {
        const bool row_in = row < a.rows;
        constexpr int kPer = kBlock == 16 ? 4 : 8;
        const int32_t loops = (a.words * kPer + 511) / 512;
        const T* base = static_cast<const T*>(a.x);
        const T* end = base + (a.rows - 1) * a.ld_x + a.cols;
        const T* x = base + (row_in ? row * a.ld_x : 0) + threadIdx.x * 16;
        auto left = [&](int32_t i) {
            return static_cast<int32_t>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(16), a.cols - (static_cast<int64_t>(i) * 512 + threadIdx.x) * 16)));
        };
        Sixteen<T> v;
        float inv_row = 1.f;
        bool finite = true;
        if constexpr (kBlock == 16) {
            uint32_t m = 0;
            for (int32_t i = 0; i < loops && row_in; ++i) {
                load16<T, kWide>(v, x + static_cast<int64_t>(i) * 512 * 16, left(i), base, end);
                m = max(m, v.largest());
            }
            m = group_max<512>(m, slot[turn]);
            finite = m < kInfBits;
            const int e = finite ? row_exponent(m) : 0;
            inv_row = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            if (row_in && threadIdx.x == 0) a.scale[row] = finite ? __uint_as_float(static_cast<uint32_t>(127 + e) << 23) : __uint_as_float(0x7fffffffu);
        }
        for (int32_t i = 0; i < loops; ++i) {
            const int32_t chunk = i * 512 + threadIdx.x;
            load16<T, kWide>(v, x + static_cast<int64_t>(i) * 512 * 16, row_in ? left(i) : 0, base, end);
            store16<T, kBlock, 512>(v, chunk, finite, inv_row, row_in && chunk < a.chunks ? a.q + row * a.ld_q + static_cast<int64_t>(chunk) * 8 : nullptr,
                                    row_in && chunk_has_scale<kBlock>(a, chunk),
                                    chunk_has_word<kBlock>(a, chunk) ? reinterpret_cast<uint32_t*>(a.block_scale + scale_word_at(row, chunk / kPer, a.words))
                                                                     : nullptr);
        }
    }
}

// ---------------------------------------------------------------- reading back

struct Fp4DequantizeArgs {
    const uint8_t* q;
    const uint8_t* block_scale;
    const float* scale;  // NULL: 1
    void* y;
    int64_t rows, ld_q, ld_y;
    int32_t cols, words;
};

// Both products a * b, each between fp32's neighbours of it rounded to the one
// whose last bit is odd (an exact one stays): what is then rounded to fewer bits is
// rounded as the exact product would be.
__device__ __forceinline__ float2 mul2_odd(float2 a, float2 b) {
    float2 lo, hi;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%4, %5};\n\tmov.b64 y, {%6, %7};\n\tmul.rm.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t"
        "mul.rp.f32x2 z, x, y;\n\tmov.b64 {%2, %3}, z;\n\t}"
        : "=f"(lo.x), "=f"(lo.y), "=f"(hi.x), "=f"(hi.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return make_float2(__float_as_uint(lo.x) & 1u ? lo.x : hi.x, __float_as_uint(lo.y) & 1u ? lo.y : hi.y);
}

// A code times an E8M0 scale of 2^126 or 2^127 may leave fp32's range where the row
// scale brings it back: an eighth of the one then goes with eight times the other
// (of a row scale so large that eight times it overflow, every product does).
__device__ __forceinline__ void keep_range(uint32_t byte, float& b, float& s) {
    if (byte > 252u) {
        b *= 0.125f;
        if (fabsf(s) < 0x1p125f) s *= 8.f;
    }
}

// The values of 16 codes in a row whose scale is no power of two, for 16-bit
// outputs. Not inlined: its registers would take a block from the SM.
template <typename T>
__device__ __noinline__ Sixteen<T> rounded16(uint2 codes, float b, float s) {
    uint32_t h[2][4];
    from_e2m1x8(codes.x, h[0]);
    from_e2m1x8(codes.y, h[1]);
    Sixteen<T> v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = mul2_odd(mul2(unpack2<__half>(h[i >> 2][i & 3]), make_float2(b, b)), make_float2(s, s));
        v.w[i] = pack2<T>(f.x, f.y);
    }
    return v;
}

// Blocks an SM holds at least: registers for more spill, and fewer leave HBM waiting.
// Rows off their boundaries, 3 and 2: 1000000 x 300 f32, block 16, 299 and 319 us;
// 262144 x 1023 f32, block 32, 282 and 273.
template <typename T, int kBlock>
__host__ __device__ constexpr int fp4_read_blocks(bool wide) { return wide ? 4 : sizeof(T) == 4 && kBlock == 32 ? 2 : 3; }

// y = code * block scale * row scale, rounded once. A code times its block scale
// has at most six bits, so with a row scale that is a power of two (the
// quantisation gives no others) the product in fp32 is exact wherever a 16-bit
// rounding could tell. Rows with other scales take a branch of their own
// (5000000 x 128 bf16, block 16: 258 us, the branch 260; 262144 x 1023: 152 and 184).
// kGroup threads of a row take 16 elements each; kFlight of a thread's pieces are
// loaded together, of kFlight rows (kRowsAhead, short rows) or of one. Bound by HBM;
// rows off their boundaries by the instructions that join and shift pieces
// (262144 x 1023 bf16: 152 us, HBM at 52 % of its rate; 262144 x 1024: 113).
template <typename T, int kBlock, bool kWide, int kGroup, bool kRowsAhead>
__global__ void __launch_bounds__(256, fp4_read_blocks<T, kBlock>(kWide)) fp4_dequantize_kernel(const Fp4DequantizeArgs a) {
    constexpr int kRows = 256 / kGroup, kFlight = 4;
    const int t = threadIdx.x % kGroup;
    const int32_t chunks = (a.cols >> 4) + ((a.cols & 15) != 0);
    const int64_t row_step = static_cast<int64_t>(gridDim.x) * kRows, first = static_cast<int64_t>(blockIdx.x) * kRows;
    // all of a block's threads stay together
    for (int64_t r0 = first; r0 < a.rows; r0 += kRowsAhead ? kFlight * row_step : row_step) {
        const int64_t row0 = r0 + threadIdx.x / kGroup;
        for (int32_t c0 = 0; c0 < chunks; c0 += kRowsAhead ? kGroup : kFlight * kGroup) {
            uint2 codes[kFlight];
            uint32_t byte[kFlight];
            float s[kFlight];
#pragma unroll
            for (int j = 0; j < kFlight; ++j) {
                const int64_t row = kRowsAhead ? row0 + j * row_step : row0;
                const int32_t chunk = c0 + t + (kRowsAhead ? 0 : j * kGroup), block = kBlock == 16 ? chunk : chunk >> 1;
                codes[j] = make_uint2(0, 0);
                byte[j] = 0;
                s[j] = 1.f;
                if (row >= a.rows || chunk >= chunks) continue;
                codes[j] = __ldg(reinterpret_cast<const uint2*>(a.q + row * a.ld_q + static_cast<int64_t>(chunk) * 8));
                byte[j] = __ldg(a.block_scale + scale_word_at(row, block >> 2, a.words) + (block & 3));
                if (a.scale) s[j] = __ldg(a.scale + row);
            }
#pragma unroll
            for (int j = 0; j < kFlight; ++j) {
                const int64_t row = kRowsAhead ? row0 + j * row_step : row0;
                const int32_t chunk = c0 + t + (kRowsAhead ? 0 : j * kGroup);
                const bool in = row < a.rows && chunk < chunks;
                float b = block_scale_value<kBlock>(byte[j]), row_s = s[j];
                if constexpr (kBlock == 32) keep_range(byte[j], b, row_s);
                Sixteen<T> v;
                bool whole = true;
                if constexpr (sizeof(T) == 2) {
                    whole = (__float_as_uint(row_s) & 0x7fffffu) == 0;
                    if (!whole) v = rounded16<T>(codes[j], b, row_s);
                }
                if (whole) {
                    uint32_t h[2][4];
                    from_e2m1x8(codes[j].x, h[0]);
                    from_e2m1x8(codes[j].y, h[1]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        // code * b first: its product with the row scale is the only one that may round
                        const float2 f = mul2(mul2(unpack2<__half>(h[i >> 2][i & 3]), make_float2(b, b)), make_float2(row_s, row_s));
                        if constexpr (sizeof(T) == 4) {
                            v.w[2 * i] = __float_as_uint(f.x);
                            v.w[2 * i + 1] = __float_as_uint(f.y);
                        } else {
                            v.w[i] = pack2<T>(f.x, f.y);
                        }
                    }
                }
                const int64_t at = static_cast<int64_t>(chunk) * 16;
                T* to = static_cast<T*>(a.y) + (in ? row * a.ld_y + at : 0);
                const int64_t left = in ? a.cols - at : 0;
                if constexpr (kWide) {
                    if (left >= 16) v.store(to);
                    else if (left > 0) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < left) to[i] = v.element(i);
                    }
                } else {
                    v.template store_any<(kGroup < 32 ? kGroup : 32)>(to, static_cast<int>(min(left, static_cast<int64_t>(1) << 20)));
                }
            }
        }
    }
}

}  // namespace maxsim
