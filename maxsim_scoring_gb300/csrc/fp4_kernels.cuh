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
    // the first n elements from p, one by one
    __device__ __forceinline__ void load_some(const T* p, int n) {
        clear();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < n) set(i, bits_of(p + i));
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(w[i]);
        } else {
            const uint32_t h = (i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu;
            if constexpr (std::is_same_v<T, __half>) return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
            else return __uint_as_float(h << 16);
        }
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

// Codes of 16 elements, and their block's scale byte.
//  block 16: with y = x / s (exact, s a power of two), b = max(e4m3(max |y| / 6), 2^-9), code = e2m1(y / b).
//  A quotient within a rounding of a code's border would change the code, so it
//  is the rounded quotient that is converted: y * (1 / b) corrected by its
//  residual (Markstein 1990: the correctly rounded reciprocal and one fma each
//  for residual and correction give the correctly rounded quotient). A rounded
//  quotient never sits on a border that the exact one is off: borders times b
//  have at most seven bits, and a 24-bit y next to one is further away than
//  half a step of the quotient. Nor does max |y| / 6 for the borders of E4M3.
//  block 32: b = 2^(floor(log2 max |x|) - 2), at least 2^-127; x / b is exact.
template <typename T, int kBlock>
__device__ __forceinline__ uint2 code16(const Sixteen<T>& v, uint32_t block_max, float inv_row, uint32_t* byte) {
    float y[16];
    if constexpr (kBlock == 16) {
        const uint32_t c = max(to_e4m3(__fdiv_rn(__uint_as_float(block_max) * inv_row, 6.f)), 1u);
        const float b = from_e4m3(c), r = __frcp_rn(b);
        *byte = c;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = v.get(i) * inv_row, q = x * r;
            y[i] = __fmaf_rn(__fmaf_rn(q, b, -x), -r, q);  // signs such that -0 stays -0
        }
    } else {
        const uint32_t field = block_max >> 23, c = field > 2 ? field - 2 : 0;
        *byte = c;
        const float inv = __uint_as_float((254u - c) << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = v.get(i) * inv;
    }
    return make_uint2(to_e2m1x8(y), to_e2m1x8(y + 8));
}

// One chunk's codes and its share of the row's scale word; the word itself is
// gathered from the lanes of the row's neighbouring chunks (kGroup lanes hold
// consecutive chunks) and stored by the first of them.
template <typename T, int kBlock, int kGroup>
__device__ __forceinline__ void store16(const Fp4QuantizeArgs& a, const Sixteen<T>& v, int64_t row, int32_t chunk, bool row_in,
                                        bool finite, float inv_row) {
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
    const bool in = row_in && chunk < a.chunks;
    if (in) *reinterpret_cast<uint2*>(a.q + row * a.ld_q + static_cast<int64_t>(chunk) * 8) = codes;
    constexpr int kPer = kBlock == 16 ? 4 : 8;  // chunks of a word
    const bool has_scale = row_in && static_cast<int64_t>(chunk) * 16 < a.cols && (kBlock == 16 || (chunk & 1) == 0);
    uint32_t word = has_scale ? byte << (kBlock == 16 ? (chunk & 3) * 8 : ((chunk >> 1) & 3) * 8) : 0u;
#pragma unroll
    for (int o = 1; o < kPer && o < kGroup; o <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
    const int32_t j = chunk / kPer;
    if (chunk % kPer == 0 && j < a.words)
        *reinterpret_cast<uint32_t*>(a.block_scale + scale_word_at(row, j, a.words)) = word;
}

// Loads the chunk of each lane. kWide: rows on 32-byte boundaries. Otherwise
// the lanes of a group (at most a warp's) load the elements of their chunks
// side by side and pass them on through shared memory: kSpan chunks, one
// element of padding for each.
template <typename T, bool kWide, int kGroup>
__device__ __forceinline__ void load16(Sixteen<T>& v, const T* row, bool row_in, int32_t chunk, int32_t cols, T* stage) {
    if constexpr (kWide) {
        const int64_t at = static_cast<int64_t>(chunk) * 16;
        if (!row_in || at >= cols) v.clear();
        else if (at + 16 <= cols) v.load(row + at);
        else v.load_some(row + at, static_cast<int>(cols - at));
    } else {
        constexpr int kLanes = kGroup < 32 ? kGroup : 32;
        const int l = static_cast<int>(threadIdx.x) % kLanes;
        T* mine = stage + (threadIdx.x - l) * 17;
        const int64_t first = static_cast<int64_t>(chunk - l) * 16;  // of the span of this group's lanes
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int e = i * kLanes + l;
            const int64_t at = first + e;
            mine[e + (e >> 4)] = row_in && at < cols ? row[at] : from_f32<T>(0.f);
        }
        __syncwarp();
        v.clear();
#pragma unroll
        for (int i = 0; i < 16; ++i) v.set(i, Sixteen<T>::bits_of(mine + l * 17 + i));
    }
}

__host__ __device__ constexpr int fp4_threads(int group) { return group < 256 ? 256 : group; }

// A row's 16-element chunks lie in the registers of a group of kGroup threads,
// kChunks each, between the row's maximum (block 16 needs it before the first
// code) and the codes: x is read once. Bound by HBM.
template <typename T, int kBlock, bool kWide, int kGroup, int kChunks>
__global__ void __launch_bounds__(fp4_threads(kGroup)) fp4_quantize_kernel(const Fp4QuantizeArgs a) {
    constexpr int kThreads = fp4_threads(kGroup), kRows = kThreads / kGroup;
    __shared__ uint32_t slot[2][kThreads / 32];
    __shared__ T stage[kWide ? 1 : kThreads * 17];
    const int t = threadIdx.x % kGroup;
    const int64_t padded = (a.rows + 127) / 128 * 128;
    int turn = 0;
    // a block's rows are all of a tile's or none, so its threads stay together
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < padded; r0 += static_cast<int64_t>(gridDim.x) * kRows, turn ^= 1) {
        const int64_t row = r0 + threadIdx.x / kGroup;
        const bool row_in = row < a.rows;
        const T* x = static_cast<const T*>(a.x) + (row_in ? row * a.ld_x : 0);
        Sixteen<T> v[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) load16<T, kWide, kGroup>(v[c], x, row_in, c * kGroup + t, a.cols, stage);
        float inv_row = 1.f;
        bool finite = true;
        if constexpr (kBlock == 16) {
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) m = max(m, v[c].largest());
            if constexpr (kGroup <= 32) {
                m = group_max<kGroup>(m, nullptr);
            } else {  // groups of a block's warps
                m = __reduce_max_sync(0xffffffffu, m);
                if ((threadIdx.x & 31) == 0) slot[turn][threadIdx.x >> 5] = m;
                __syncthreads();
                const int first = static_cast<int>(threadIdx.x) / kGroup * (kGroup / 32);
                m = __reduce_max_sync(0xffffffffu, slot[turn][first + (threadIdx.x & 31) % (kGroup / 32)]);
            }
            finite = m < kInfBits;
            const int e = finite ? row_exponent(m) : 0;
            inv_row = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            if (row_in && t == 0) a.scale[row] = finite ? __uint_as_float(static_cast<uint32_t>(127 + e) << 23) : __uint_as_float(0x7fffffffu);
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
            store16<T, kBlock, kGroup>(a, v[c], row, c * kGroup + t, row_in, finite, inv_row);
    }
}

// Rows that no group holds: a block per row, read twice with block 16.
template <typename T, int kBlock, bool kWide>
__global__ void __launch_bounds__(512) fp4_quantize_long_kernel(const Fp4QuantizeArgs a) {
    __shared__ uint32_t slot[2][16];
    __shared__ T stage[kWide ? 1 : 512 * 17];
    const int64_t padded = (a.rows + 127) / 128 * 128;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < padded; row += gridDim.x, turn ^= 1) {
        const bool row_in = row < a.rows;
        const T* x = static_cast<const T*>(a.x) + (row_in ? row * a.ld_x : 0);
        const int32_t loops = (a.words * (kBlock == 16 ? 4 : 8) + 511) / 512;
        Sixteen<T> v;
        float inv_row = 1.f;
        bool finite = true;
        if constexpr (kBlock == 16) {
            uint32_t m = 0;
            for (int32_t i = 0; i < loops && row_in; ++i) {
                load16<T, kWide, 512>(v, x, row_in, i * 512 + threadIdx.x, a.cols, stage);
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
            load16<T, kWide, 512>(v, x, row_in, chunk, a.cols, stage);
            store16<T, kBlock, 512>(a, v, row, chunk, row_in, finite, inv_row);
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

// y = code * block scale * row scale, rounded once: a code times an E4M3 scale
// has at most six bits, and the row scales that the quantisation gives are
// powers of two, so 16-bit rows are exact wherever their exponents reach.
// kGroup threads of a row take 16 elements each. Bound by HBM.
template <typename T, int kBlock, bool kWide, int kGroup>
__global__ void __launch_bounds__(256) fp4_dequantize_kernel(const Fp4DequantizeArgs a) {
    constexpr int kRows = 256 / kGroup;
    const int t = threadIdx.x % kGroup;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kGroup; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * kRows) {
        const float s = a.scale ? a.scale[row] : 1.f;
        T* y = static_cast<T*>(a.y) + row * a.ld_y;
        for (int32_t chunk = t; chunk < (a.cols >> 4) + ((a.cols & 15) != 0); chunk += kGroup) {
            const uint2 codes = __ldg(reinterpret_cast<const uint2*>(a.q + row * a.ld_q + static_cast<int64_t>(chunk) * 8));
            const int32_t block = kBlock == 16 ? chunk : chunk >> 1;
            const float b = block_scale_value<kBlock>(__ldg(a.block_scale + scale_word_at(row, block >> 2, a.words) + (block & 3)));
            uint32_t h[2][4];
            from_e2m1x8(codes.x, h[0]);
            from_e2m1x8(codes.y, h[1]);
            Sixteen<T> v;
            v.clear();
            float f[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const unsigned short u = static_cast<unsigned short>(h[i >> 3][(i & 7) >> 1] >> ((i & 1) * 16));
                f[i] = __half2float(__ushort_as_half(u)) * b * s;
            }
            const int64_t at = static_cast<int64_t>(chunk) * 16;
            const int n = static_cast<int>(min(static_cast<int64_t>(16), a.cols - at));
            T* to = y + at;
            if (kWide && n == 16) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const T o = from_f32<T>(f[i]);
                    v.set(i, Sixteen<T>::bits_of(&o));
                }
                v.store(to);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i < n) to[i] = from_f32<T>(f[i]);
            }
        }
    }
}

}  // namespace maxsim
