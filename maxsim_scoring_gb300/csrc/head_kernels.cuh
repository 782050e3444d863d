// Row quantisation to INT8 and dropout (the token head's elementwise
// operators).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

namespace maxsim {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// ---------------------------------------------------------------- row quantisation
//
// The scale, a 127th of max |x|, needs the whole row before the first code, so a
// row is held in registers between the two: one read of x, one write of q. A
// row belongs to a group of 1, 8, 32, 128 or 512 threads, each holding up to
// kChunks 16-byte chunks (or single elements, see RowMode); only rows beyond that
// are read twice. Several short rows share a warp: fewer shuffle steps for a row,
// and their loads are in flight together.
// Bound by HBM: 5,000,000 x 128 f32 in 480 us (6.7 TB/s), 65536 x 4096 bf16 in
// 121 us (6.6 TB/s); 16-bit rows of 128 with the norm in 220 us for 3,000,000 (5.3
// TB/s, 70 % of the issue slots), rows off their 16-byte boundaries by the
// handling of their ends or by single elements (100000 x 1023 bf16 in 90 us, 3.4
// TB/s, f32 in 102 us, 5.0 TB/s).

// Maximum of two pairs of unsigned 16-bit values.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// One chunk of a row: kVec elements, 16 bytes or a single one.
template <typename T, bool kWide>
struct Chunk;

template <typename T>
struct Chunk<T, true> {
    static constexpr int kVec = 16 / static_cast<int>(sizeof(T));
    uint4 v;
    __device__ __forceinline__ void load(const T* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
    // elements first .. last - 1 from p one by one, zeros around them
    __device__ __forceinline__ void load_some(const T* p, int first, int last) {
        alignas(16) T e[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) e[i] = i >= first && i < last ? p[i] : from_f32<T>(0.f);
        v = *reinterpret_cast<const uint4*>(e);
    }
    // zeros outside elements first .. last - 1
    __device__ __forceinline__ void keep(int first, int last) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        constexpr int kPer = 4 / static_cast<int>(sizeof(T));  // elements of a word
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t m = i * kPer >= first && i * kPer < last ? (kPer == 1 ? 0xffffffffu : 0xffffu) : 0u;
            if (kPer == 2 && i * 2 + 1 >= first && i * 2 + 1 < last) m |= 0xffff0000u;
            w[i] &= m;
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(w[i]);
        } else {
            const unsigned short h = static_cast<unsigned short>((i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu);
            if constexpr (std::is_same_v<T, __half>) return __half2float(__ushort_as_half(h));
            else return __uint_as_float(static_cast<uint32_t>(h) << 16);
        }
    }
    // max |.| so far, as bit patterns (ordered as the values; infinities and NaN on top)
    __device__ __forceinline__ uint32_t fold_max(uint32_t m) const {
        if constexpr (sizeof(T) == 4) {
            return max(max(m, max(v.x & 0x7fffffffu, v.y & 0x7fffffffu)),
                       max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
        } else {
            return max_u16x2(max_u16x2(m, max_u16x2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu)),
                             max_u16x2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
        }
    }
    static __device__ __forceinline__ uint32_t max_bits(uint32_t m) {
        return sizeof(T) == 4 ? m : max(m >> 16, m & 0xffffu);
    }
    static __device__ __forceinline__ void store(int8_t* q, const uint32_t* w) {
        if constexpr (sizeof(T) == 4) *reinterpret_cast<uint32_t*>(q) = w[0];
        else *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    }
};

template <typename T>
struct Chunk<T, false> {
    static constexpr int kVec = 1;
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void clear() { v = from_f32<T>(0.f); }
    __device__ __forceinline__ float get(int) const { return to_f32(v); }
    __device__ __forceinline__ uint32_t bits() const {
        if constexpr (sizeof(T) == 4) return __float_as_uint(v) & 0x7fffffffu;
        else return *reinterpret_cast<const unsigned short*>(&v) & 0x7fffu;
    }
    __device__ __forceinline__ uint32_t fold_max(uint32_t m) const { return max(m, bits()); }
    static __device__ __forceinline__ uint32_t max_bits(uint32_t m) { return m; }
    static __device__ __forceinline__ void store(int8_t* q, const uint32_t* w) { *q = static_cast<int8_t>(w[0]); }
};

// From the largest |x| of a row (bits of T): whether the row is finite, and s = max(a * (1 / 127), 2^-126).
template <typename T>
__device__ __forceinline__ bool row_step(uint32_t bits, float* s) {
    float a;
    bool finite;
    if constexpr (sizeof(T) == 4) {
        finite = bits < 0x7f800000u;
        a = __uint_as_float(bits);
    } else if constexpr (std::is_same_v<T, __half>) {
        finite = bits < 0x7c00u;
        a = __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
    } else {
        finite = bits < 0x7f80u;
        a = __uint_as_float(bits << 16);
    }
    *s = finite ? fmaxf(__fmul_rn(a, 1.f / 127.f), FLT_MIN) : 1.f;
    return finite;
}

// The codes of one chunk, packed in w, and with kNorm its sum of squares of x / s.
// rint(x / s) wants an IEEE division per element. x * inv, inv = 1 / s, is at
// most 1.2e-5 away from the rounded quotient (|x / s| <= 127: 2^-24 relative
// from inv, half a unit of the last place from the division), so only
// products within 3e-5 of a half-integer can round to another code, and only
// chunks that hold such a product divide. The product is rounded to an integer
// by adding 1.5 * 2^23 in the same fma; the sum's low byte is the code.
template <typename T, bool kWide, bool kNorm>
__device__ __forceinline__ float code_chunk(const Chunk<T, kWide>& c, float s, float inv, uint32_t keep, uint32_t* w) {
    constexpr float kMagic = 12582912.f;
    constexpr int kVec = Chunk<T, kWide>::kVec;
    uint32_t m[kVec];
    float sum = 0.f, off = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const float x = c.get(i);
        const float r = __fmaf_rn(x, inv, kMagic);
        off = fmaxf(off, fabsf(__fmaf_rn(x, inv, -(r - kMagic))));
        m[i] = __float_as_uint(r);
        if constexpr (kNorm) {
            const float y = x * inv;
            sum = __fmaf_rn(y, y, sum);
        }
    }
    if (off > 0.49997f) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) m[i] = __float_as_uint(__fdiv_rn(c.get(i), s) + kMagic);
    }
    if constexpr (kVec == 1) {
        w[0] = m[0] & keep;
    } else {
#pragma unroll
        for (int i = 0; i < kVec / 4; ++i) {
            const uint32_t lo = __byte_perm(m[4 * i], m[4 * i + 1], 0x0040), hi = __byte_perm(m[4 * i + 2], m[4 * i + 3], 0x0040);
            w[i] = __byte_perm(lo, hi, 0x5410) & keep;
        }
    }
    return sum;
}

template <bool kNorm>
__device__ __forceinline__ float row_scale(bool finite, float s, float sum) {
    float out = s;
    if constexpr (kNorm) out = sum > 0.f ? rsqrtf(sum) : FLT_MIN;
    return finite ? out : __uint_as_float(0x7fffffffu);
}

// Sum and maximum over a group of kGroup threads, the same in all of them.
// Groups above a warp are blocks; `slot` is shared memory for one value per
// warp and must not be in use (two alternate).
template <int kGroup>
__device__ __forceinline__ uint32_t group_max(uint32_t v, uint32_t* slot) {
    if constexpr (kGroup >= 32) v = __reduce_max_sync(0xffffffffu, v);
    else
#pragma unroll
        for (int o = kGroup / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    if constexpr (kGroup > 32) {
        if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
        __syncthreads();
        v = __reduce_max_sync(0xffffffffu, slot[(threadIdx.x & 31) % (kGroup / 32)]);
    }
    return v;
}

template <int kGroup>
__device__ __forceinline__ float group_sum(float v, float* slot) {
#pragma unroll
    for (int o = (kGroup < 32 ? kGroup : 32) / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (kGroup > 32) {
        if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < kGroup / 32; ++i) v += slot[i];
    }
    return v;
}

struct QuantizeArgs {
    const void* x;
    int8_t* q;
    float* scale;
    int64_t rows, ld_x, ld_q;
    int32_t cols;
};

// How rows are read: element by element; in 16-byte chunks from their starts
// (rows on 16-byte boundaries); or in the aligned chunks that they touch, whose
// elements of other rows count as zeros and are not stored (rows anywhere, if
// the codes of a chunk are an aligned piece of q too: the phases of x and q agree).
enum RowMode { kSingle, kWhole, kTouched };

template <typename T, RowMode kMode>
struct QuantizeRow {
    using C = Chunk<T, kMode != kSingle>;
    const T* x;
    int8_t* q;
    int64_t before, after;  // elements of the operand in front of the row and from its start on
    int32_t cols, skip;     // skip: elements of the first chunk that are not the row's

    __device__ __forceinline__ QuantizeRow(const QuantizeArgs& a, int64_t r) {
        before = r * a.ld_x;
        after = (a.rows - 1 - r) * a.ld_x + a.cols;
        x = static_cast<const T*>(a.x) + before;
        q = a.q + r * a.ld_q;
        cols = a.cols;
        skip = kMode == kTouched ? static_cast<int32_t>(reinterpret_cast<uintptr_t>(x) / sizeof(T)) & (C::kVec - 1) : 0;
    }
    template <typename I>
    __device__ __forceinline__ I col(I chunk) const { return chunk * C::kVec - skip; }
    template <typename I>
    __device__ __forceinline__ void load(C& c, I chunk, bool start) const {  // start: may hold the row's first element
        const I at = col(chunk);
        if (at >= cols) {
            c.clear();
        } else if constexpr (kMode != kTouched) {
            c.load(x + at);
        } else if ((!start || at >= 0) && at + C::kVec <= cols) {
            c.load(x + at);
        } else {
            const int first = start && at < 0 ? static_cast<int>(-at) : 0, last = static_cast<int>(min(static_cast<I>(C::kVec), cols - at));
            if (before + at >= 0 && at + C::kVec <= after) {
                c.load(x + at);
                c.keep(first, last);
            } else {  // not past the operand's ends
                c.load_some(x + at, first, last);
            }
        }
    }
    template <typename I>
    __device__ __forceinline__ void store(const uint32_t* w, I chunk, bool start) const {
        const I at = col(chunk);
        if (at >= cols) return;
        if constexpr (kMode != kTouched) {
            C::store(q + at, w);
        } else if ((!start || at >= 0) && at + C::kVec <= cols) {
            C::store(q + at, w);
        } else {
#pragma unroll
            for (int i = 0; i < C::kVec; ++i)
                if ((!start || at + i >= 0) && at + i < cols) q[at + i] = static_cast<int8_t>(w[i / 4] >> (8 * (i % 4)));
        }
    }
};

__host__ __device__ constexpr int quantize_threads(int group) { return group > 128 ? group : 128; }

// Blocks of an SM that registers must leave room for: with few single elements a
// thread, all of its threads (500000 x 30 f32 23.7 us, and 26 with 34 registers).
// 0: none in particular.
__host__ __device__ constexpr int quantize_blocks(RowMode mode, int chunks) { return mode == kSingle && chunks <= 4 ? 16 : 0; }

template <typename T, RowMode kMode, bool kNorm, int kGroup, int kChunks>
__global__ void __launch_bounds__(quantize_threads(kGroup), quantize_blocks(kMode, kChunks))
quantize_rows_kernel(const QuantizeArgs a) {
    using C = typename QuantizeRow<T, kMode>::C;
    constexpr int kThreads = quantize_threads(kGroup), kPerBlock = kThreads / kGroup;
    __shared__ uint32_t s_max[16];
    __shared__ float s_sum[16];
    const int g = threadIdx.x / kGroup, t = threadIdx.x % kGroup;
    // every thread of the block walks the same number of rows: the groups reduce with full-warp shuffles
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kPerBlock; r0 < a.rows;
         r0 += static_cast<int64_t>(gridDim.x) * kPerBlock) {
        const int64_t r = r0 + g;
        const bool real = r < a.rows;
        const QuantizeRow<T, kMode> row(a, real ? r : r0);
        C c[kChunks];
#pragma unroll
        for (int j = 0; j < kChunks; ++j) row.load(c[j], j * kGroup + t, j == 0);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) m = c[j].fold_max(m);
        m = group_max<kGroup>(C::max_bits(m), s_max);
        float s;
        const bool finite = row_step<T>(m, &s);
        const float inv = __frcp_rn(s);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            if (kGroup == 1 && row.col(j) >= a.cols) continue;
            uint32_t w[2];
            sum += code_chunk<T, kMode != kSingle, kNorm>(c[j], s, inv, finite ? 0xffffffffu : 0u, w);
            if (real) row.store(w, j * kGroup + t, j == 0);
        }
        if constexpr (kNorm) sum = group_sum<kGroup>(sum, s_sum);
        if (real && t == 0) a.scale[r] = row_scale<kNorm>(finite, s, sum);
        if constexpr (kGroup > 32) __syncthreads();  // the slots are free again
    }
}

// Rows too long for the registers of a block: read once for the maximum, once for the codes.
template <typename T, RowMode kMode, bool kNorm>
__global__ void __launch_bounds__(512) quantize_long_rows_kernel(const QuantizeArgs a) {
    using C = typename QuantizeRow<T, kMode>::C;
    __shared__ uint32_t s_max[16];
    __shared__ float s_sum[16];
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const QuantizeRow<T, kMode> row(a, r);
        uint32_t m = 0;
#pragma unroll 4
        for (int64_t i = threadIdx.x; row.col(i) < a.cols; i += 512) {
            C c;
            row.load(c, i, true);
            m = c.fold_max(m);
        }
        m = group_max<512>(C::max_bits(m), s_max);
        float s;
        const bool finite = row_step<T>(m, &s);
        const float inv = __frcp_rn(s);
        float sum = 0.f;
#pragma unroll 4
        for (int64_t i = threadIdx.x; row.col(i) < a.cols; i += 512) {
            C c;
            row.load(c, i, true);
            uint32_t w[2];
            sum += code_chunk<T, kMode != kSingle, kNorm>(c, s, inv, finite ? 0xffffffffu : 0u, w);
            row.store(w, i, true);
        }
        if constexpr (kNorm) sum = group_sum<512>(sum, s_sum);
        if (threadIdx.x == 0) a.scale[r] = row_scale<kNorm>(finite, s, sum);
        __syncthreads();
    }
}

// ---------------------------------------------------------------- dropout

// Philox4x32-10 (Salmon et al. 2011): ten rounds of two 32 x 32 -> 64 bit
// products, the key stepped by the Weyl constants.
__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = static_cast<uint64_t>(c.x) * 0xD2511F53u, b = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
        c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k0, static_cast<uint32_t>(b),
                       static_cast<uint32_t>(a >> 32) ^ c.w ^ k1, static_cast<uint32_t>(a));
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

struct DropoutArgs {
    const void* x;
    const void* residual;  // NULL = none
    void* y;
    int64_t rows, ld_x, ld_r, ld_y;
    int64_t n;              // rows * cols
    int32_t cols;
    uint32_t drop;          // T: elements that draw less than this are dropped
    float scale;
    uint32_t key0, key1, off0, off1;
    uint32_t div_mul, div_shift;  // i / d = (i * div_mul) >> (32 + div_shift) for i < 2^31 (d: see the kernels)
};

// i / d by a product (d's reciprocal rounded up to 32 bits), for 0 <= i < 2^31.
__device__ __forceinline__ uint32_t fast_div(uint32_t i, uint32_t mul, uint32_t shift) {
    return shift == 0xffffffffu ? i : __umulhi(i, mul) >> shift;
}

__device__ __forceinline__ uint4 draw_block(const DropoutArgs& a, int64_t b) {
    return philox4x32_10(make_uint4(static_cast<uint32_t>(b), static_cast<uint32_t>(static_cast<uint64_t>(b) >> 32),
                                    a.off0, a.off1),
                         a.key0, a.key1);
}

// Two 16-bit values of T in a word, and one of them again.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <typename T>
__device__ __forceinline__ T half_of(uint32_t w, int i) {
    const unsigned short h = static_cast<unsigned short>(i ? w >> 16 : w);
    return *reinterpret_cast<const T*>(&h);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (std::is_same_v<T, __half>) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <typename T>
struct Eight {  // eight consecutive elements
    static constexpr int kWords = 4 * static_cast<int>(sizeof(T)) / 2;
    uint32_t v[kWords];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
            v[i] = w.x; v[i + 1] = w.y; v[i + 2] = w.z; v[i + 3] = w.w;
        }
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < kWords; i += 4)
            *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(p) + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
    // element e: p[e], or past a row's end (e >= end) q[e]
    __device__ __forceinline__ void gather(const T* p, const T* q, int end) {
        T t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = (i >= end ? q : p)[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[i] = __float_as_uint(t[i]);
            } else {
                const uint32_t h = *reinterpret_cast<const unsigned short*>(&t[i]);
                v[i / 2] = (i & 1) ? v[i / 2] | h << 16 : h;
            }
        }
    }
    __device__ __forceinline__ float2 pair(int i) const {
        if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
        else return unpack2<T>(v[i]);
    }
    __device__ __forceinline__ void set_pair(int i, float a, float b) {
        if constexpr (sizeof(T) == 4) {
            v[2 * i] = __float_as_uint(a);
            v[2 * i + 1] = __float_as_uint(b);
        } else {
            v[i] = pack2<T>(a, b);
        }
    }
};

enum { kXFlat = 0, kXRows = 1, kXGather = 2 };

// Dropout by pieces of eight elements that share a counter, 16 bytes (f32: 32)
// of y and the residual: one read, one write and ten rounds of Philox a piece.
//  kXFlat: x, residual and y are each one run of n elements.
//  kXRows: cols is a multiple of 8 and the rows of all three start on 16-byte
//          boundaries; fast_div divides a piece's number by the pieces of a row.
//  kXGather: residual and y are runs; x's rows lie apart or off their
//          boundaries (cols >= 8), and its elements are loaded one by one;
//          fast_div divides by cols. (Paths of their own for whole pieces and for
//          4-byte aligned ones left 16384 x 1023 at 26 us and took 1000000 x 101
//          from 139 to 174; one piece a thread instead of two: 22 and 121.)
// A warp takes 32 * kPieces neighbouring pieces at a time, so that several
// loads of a thread are in flight and a warp's accesses stay close together
// (262144 x 1024 f16 without residual: 183 us with a thread's two pieces a grid
// apart, 172 with two neighbouring, 171 with four; with a bf16 residual 264, 247
// and 238). Bound by HBM, if the arithmetic stays near 100 instructions a
// piece (three rounds of Philox instead of ten: 163 us): the comparisons take
// the drawn halves as they lie in their words, and results are rounded two at
// a time.
template <typename T, int kX>
__host__ __device__ constexpr int dropout_pieces() { return kX == kXGather ? 1 : sizeof(T) == 2 ? 4 : 2; }

template <typename T, int kX, bool kRes>
__global__ void __launch_bounds__(256) dropout_wide_kernel(const DropoutArgs a) {
    constexpr int kPieces = dropout_pieces<T, kX>();
    const T* x = static_cast<const T*>(a.x);
    const T* res = static_cast<const T*>(a.residual);
    T* y = static_cast<T*>(a.y);
    const int64_t blocks = a.n >> 3;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 256 * kPieces;
    const int64_t first = blockIdx.x * static_cast<int64_t>(256 * kPieces) + (threadIdx.x >> 5) * (32 * kPieces) + (threadIdx.x & 31);
    const bool some = a.drop < 65536u;                 // anything is kept
    const uint32_t least = a.drop << 16;
    for (int64_t b0 = first; b0 < blocks; b0 += step) {
        Eight<T> xv[kPieces], rv[kPieces];
        int64_t at_y[kPieces];
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int64_t b = b0 + j * 32;
            if (b >= blocks) break;
            const int64_t i = b << 3;
            int64_t at_r = i;
            at_y[j] = i;
            if constexpr (kX == kXFlat) {
                xv[j].load(x + i);
            } else if constexpr (kX == kXRows) {
                const int32_t per_row = a.cols >> 3;
                const int64_t row = b < 0x80000000ll ? fast_div(static_cast<uint32_t>(b), a.div_mul, a.div_shift) : b / per_row;
                const int64_t col = (b - row * per_row) << 3;
                xv[j].load(x + row * a.ld_x + col);
                at_r = row * a.ld_r + col;
                at_y[j] = row * a.ld_y + col;
            } else {
                const int64_t row = i < 0x80000000ll ? fast_div(static_cast<uint32_t>(i), a.div_mul, a.div_shift) : i / a.cols;
                const int64_t gap = a.ld_x - a.cols;
                const T* p = x + i + row * gap;
                xv[j].gather(p, p + gap, static_cast<int>(min((row + 1) * a.cols - i, static_cast<int64_t>(8))));
            }
            if constexpr (kRes) rv[j].load(res + at_r);
        }
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int64_t b = b0 + j * 32;
            if (b >= blocks) break;
            const uint4 u = draw_block(a, b);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // half u >= T exactly where u << 16 (with anything below) >= T << 16
                const bool keep0 = some && (w[e] << 16) >= least, keep1 = some && w[e] >= least;
                const float2 v = xv[j].pair(e);
                float y0 = keep0 ? v.x * a.scale : 0.f, y1 = keep1 ? v.y * a.scale : 0.f;
                if constexpr (kRes) {
                    const float2 r = rv[j].pair(e);
                    y0 += r.x;
                    y1 += r.y;
                }
                xv[j].set_pair(e, y0, y1);
            }
            xv[j].store(y + at_y[j]);
        }
    }
    if (kX != kXRows && first == 0 && (a.n & 7)) {  // the short last piece
        const uint4 u = draw_block(a, blocks);
        const int64_t skip = kX == kXGather ? (a.rows - 1) * (a.ld_x - a.cols) : 0;  // it ends the last row
        for (int e = 0; e < static_cast<int>(a.n & 7); ++e) {
            const int64_t i = (blocks << 3) + e;
            const uint32_t word = e < 2 ? u.x : e < 4 ? u.y : e < 6 ? u.z : u.w;
            const uint32_t bits = (e & 1) ? word >> 16 : word & 0xffffu;
            float v = bits >= a.drop ? to_f32(x[i + skip]) * a.scale : 0.f;
            if constexpr (kRes) v += to_f32(res[i]);
            y[i] = from_f32<T>(v);
        }
    }
}

// Dropout for every other layout (residual or y with rows apart and off their
// 16-byte boundaries, or the narrowest rows). A warp takes 256 consecutive elements: its lanes draw one
// counter each, pass the bits through shared memory, and then take every
// 32nd element, so that loads and stores of single elements are coalesced.
// kWidth = 256: rows are at least as long as the run, which then crosses at
// most one row's end, and one division (fast_div by cols) places it; 0: any
// width, a division per element. Bound by instruction issue (16384 x 1023 bf16
// with a residual, all rows apart: 33 us, 3.1 TB/s).
template <typename T, bool kRes, int kWidth>
__global__ void __launch_bounds__(256) dropout_any_kernel(const DropoutArgs a) {
    __shared__ uint4 s_bits[8][32];
    const T* x = static_cast<const T*>(a.x);
    const T* res = static_cast<const T*>(a.residual);
    T* y = static_cast<T*>(a.y);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned short* bits = reinterpret_cast<const unsigned short*>(s_bits[warp]) + lane;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8 * 256;
    auto divide = [&](int64_t i) {
        return i < 0x80000000ll ? static_cast<int64_t>(fast_div(static_cast<uint32_t>(i), a.div_mul, a.div_shift)) : i / a.cols;
    };
    for (int64_t i0 = (static_cast<int64_t>(blockIdx.x) * 8 + warp) * 256; i0 < a.n; i0 += step) {
        const int left = static_cast<int>(min(a.n - i0, static_cast<int64_t>(256))) - lane;  // element 32 j exists while 32 j < left
        const int64_t row0 = kWidth ? divide(i0) : 0;
        // element c of row0 onward: at p[c], or past the row's end (c >= cols) at q[c]
        const uint32_t col0 = static_cast<uint32_t>(i0 - row0 * a.cols) + lane;  // unsigned: may reach 2^31
        const T* px = x + row0 * a.ld_x + col0;
        const T* pr = res + row0 * a.ld_r + col0;
        T* py = y + row0 * a.ld_y + col0;
        const int64_t dx = a.ld_x - a.cols, dr = a.ld_r - a.cols, dy = a.ld_y - a.cols;
        const int32_t end = static_cast<int32_t>(a.cols - col0);  // 32 j >= end: the next row
        T xv[8], rv[8];
        s_bits[warp][lane] = draw_block(a, (i0 >> 3) + lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (32 * j < left) {
                if constexpr (kWidth) {
                    xv[j] = (32 * j >= end ? px + dx : px)[32 * j];
                    if constexpr (kRes) rv[j] = (32 * j >= end ? pr + dr : pr)[32 * j];
                } else {
                    const int64_t i = i0 + 32 * j + lane, row = divide(i);
                    xv[j] = x[i + row * dx];
                    if constexpr (kRes) rv[j] = res[i + row * dr];
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (32 * j < left) {
                float v = bits[32 * j] >= a.drop ? to_f32(xv[j]) * a.scale : 0.f;
                if constexpr (kRes) v += to_f32(rv[j]);
                T* to;
                if constexpr (kWidth) {
                    to = (32 * j >= end ? py + dy : py) + 32 * j;
                } else {
                    const int64_t i = i0 + 32 * j + lane;
                    to = y + i + divide(i) * dy;
                }
                *to = from_f32<T>(v);
            }
        }
        __syncwarp();
    }
}

}  // namespace maxsim
