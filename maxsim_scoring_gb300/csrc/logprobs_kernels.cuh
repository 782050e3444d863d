// Log probabilities of given columns of score or logit rows, the rows'
// entropies and strongest columns, and the gradient.
//
// With the row's maximum M over its active columns and t_j = (x_j - M) * c,
// c = scale * log2 e:  S = sum 2^t_j, W = sum 2^t_j t_j, L = log2 S, and
//   log p_j = ln 2 * (t_j - L)      entropy = ln 2 * (L - W / S).
// The difference x_j - M is rounded once before it is scaled, so that columns
// near the maximum, which decide, keep their digits however large the scores.
#pragma once

#include <cstdint>

#include "head_kernels.cuh"
#include "ptx.cuh"
#include "tile_store.cuh"

namespace maxsim {

struct LogprobsArgs {
    const void* x;            // [rows, n], rows ld apart
    const int64_t* targets;   // [rows, T]
    const uint8_t* mask;      // NULL, or rows ld_mask apart (0: one for all)
    int64_t rows, n, ld, ld_mask;
    int32_t T, k;
    float scale, c;           // c = scale * log2 e
    float* logprob;           // [rows, T]
    float* entropy;           // [rows]
    int32_t* top_idx;         // [rows, k]
    float* top_logprob;       // [rows, k]
    float* stats;             // [rows, 2]: M and L
    int* status;
};

constexpr float kLn2 = 0.693147180559945309f;
constexpr int kLogprobsMaxTop = 64;
constexpr int kDeviceInput = 6;  // MAXSIM_ERR_DEVICE_INPUT
constexpr float kNoExponent = -1000.f;  // 2^t is 0 from here on
constexpr float kLowExponent = -65536.f;  // exponents that are not cut to kNoExponent end here
constexpr float kLargest = 0x1.fffffep127f;

__device__ __forceinline__ float exp2_fast(float t) {  // 2^-22 relative
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(t));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN where either is
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {  // both sums in one instruction
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xff800000u); }

// Bytes of ones where the selected byte's high bit is set (a selector's digit: 8 + the byte).
__device__ __forceinline__ uint32_t byte_signs(uint32_t w, uint32_t selector) {
    uint32_t d;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(d) : "r"(w), "r"(selector));
    return d;
}

// ---------------------------------------------------------------- 16-byte pieces of a row

template <typename T>
struct PieceOf {
    static constexpr int kVec = 16 / static_cast<int>(sizeof(T));
    // the type's minus infinity in every place of a word
    static constexpr uint32_t kMinusInf = std::is_same_v<T, float> ? 0xff800000u : std::is_same_v<T, __half> ? 0xfc00fc00u : 0xff80ff80u;

    // elements 2 i and 2 i + 1
    static __device__ __forceinline__ float2 pair(const uint4& u, int i) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return unpack2<T>(w[i]);
    }
    // the larger elements of two words, NaN where both are
    static __device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b) {
        uint32_t d;
        if constexpr (std::is_same_v<T, float>) asm("max.f32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        else if constexpr (std::is_same_v<T, __half>) asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        else asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    // the smaller ones
    static __device__ __forceinline__ uint32_t min_words(uint32_t a, uint32_t b) {
        uint32_t d;
        if constexpr (std::is_same_v<T, float>) asm("min.f32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        else if constexpr (std::is_same_v<T, __half>) asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        else asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ uint32_t min_words(const uint4& u) { return min_words(min_words(u.x, u.y), min_words(u.z, u.w)); }
    static __device__ __forceinline__ float word_min(uint32_t w) {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w);
        const float2 v = unpack2<T>(w);
        return fminf(v.x, v.y);
    }
    static __device__ __forceinline__ uint32_t max_words(const uint4& u) { return max_words(max_words(u.x, u.y), max_words(u.z, u.w)); }
    static __device__ __forceinline__ float word_max(uint32_t w) {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w);
        const float2 v = unpack2<T>(w);
        return fmaxf(v.x, v.y);
    }
    // minus infinity where the high bit of the element's byte in m is clear
    static __device__ __forceinline__ uint4 masked(uint4 u, const uint32_t (&m)[kVec / 4]) {
        uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // the sign of one byte (of two) in all bytes of its element
            const uint32_t keep = sizeof(T) == 4 ? byte_signs(m[0], 0x8888 + 0x1111 * i) : byte_signs(m[i >> 1], (i & 1) ? 0xbbaa : 0x9988);
            w[i] = (w[i] & keep) | (kMinusInf & ~keep);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// High bits of the bytes of w that are not zero.
__device__ __forceinline__ uint32_t nonzero_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x7f7f7f7fu) | w; }

// A row seen as aligned 16-byte pieces: piece p holds columns p * kVec - skip
// and on; the first and the last one may reach over the row's ends, and are
// read element by element then. Columns fit 32 bits.
template <typename T>
struct PiecedRow {
    using P = PieceOf<T>;
    static constexpr int kVec = P::kVec;
    const T* x;
    const uint8_t* mask;
    int32_t n, skip, pieces;
    uint32_t x_by, mask_by;  // bytes that pieces of x, and of the mask, begin behind a 16- and a kVec-byte boundary

    // `place`: pieces are those of the row that starts here (a multiple of T's size)
    __device__ __forceinline__ PiecedRow(const T* row, const uint8_t* m, int64_t cols, const T* place)
        : x(row), mask(m), n(static_cast<int32_t>(cols)) {
        skip = static_cast<int32_t>(reinterpret_cast<uintptr_t>(place) / sizeof(T)) & (kVec - 1);
        pieces = static_cast<int32_t>((cols + skip + kVec - 1) / kVec);
        x_by = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) - skip * sizeof(T)) & 15u;
        mask_by = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(m) - skip) & (kVec - 1);
    }
    // pieces around p are the row's too: the aligned pieces and mask words that hold p may be read
    __device__ __forceinline__ bool interior(int32_t p) const { return column(p) >= kVec && column(p) + 2 * kVec <= n; }
    __device__ __forceinline__ int32_t column(int32_t p) const { return p * kVec - skip; }
    __device__ __forceinline__ bool whole(int32_t p) const { return column(p) >= 0 && column(p) + kVec <= n; }
    // whole piece p
    __device__ __forceinline__ uint4 load_whole(int32_t p) const { return __ldg(reinterpret_cast<const uint4*>(x + column(p))); }
    // An interior piece of rows of another phase: the two aligned pieces that hold it, and it from them.
    __device__ __forceinline__ void load_around(int32_t p, uint4& lo, uint4& hi) const {
        const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(x + column(p)) & ~uintptr_t(15));
        lo = __ldg(q);
        hi = __ldg(q + 1);
    }
    __device__ __forceinline__ uint4 shifted(const uint4& lo, const uint4& hi) const {
        uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        if (x_by & 8u) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (x_by & 4u) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        const uint32_t bits = (x_by & 3u) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // Piece p, element by element where it is not whole or x has another phase; what is not the row's is minus infinity.
    __device__ __forceinline__ uint4 load(int32_t p) const {
        const int32_t at = column(p);
        if (at >= 0 && at + kVec <= n && x_by == 0) return load_whole(p);
        T e[kVec];  // all loads before the first use
#pragma unroll
        for (int i = 0; i < kVec; ++i) e[i] = x[min(max(at + i, 0), n - 1)];
        alignas(16) T o[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) o[i] = at + i >= 0 && at + i < n ? e[i] : from_f32<T>(minus_inf());
        return *reinterpret_cast<const uint4*>(o);
    }
    // The words that hold an interior piece's mask bytes, and from them a high bit for each active column.
    struct MaskWords {
        uint32_t v[kVec / 4 + 1];
    };
    __device__ __forceinline__ void load_mask(int32_t p, MaskWords& w) const {
        const uint8_t* from = mask + column(p);
        if (mask_by == 0) {
            if constexpr (kVec == 8) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(from));
                w.v[0] = v.x;
                w.v[1] = v.y;
            } else {
                w.v[0] = __ldg(reinterpret_cast<const uint32_t*>(from));
            }
            w.v[kVec / 4] = 0;
        } else {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(from) & ~uintptr_t(3));
#pragma unroll
            for (int i = 0; i <= kVec / 4; ++i) w.v[i] = __ldg(q + i);
        }
    }
    __device__ __forceinline__ uint4 masked(const uint4& u, const MaskWords& w) const {
        uint32_t m[kVec / 4];
#pragma unroll
        for (int i = 0; i < kVec / 4; ++i) m[i] = nonzero_bytes(__funnelshift_r(w.v[i], w.v[i + 1], (mask_by & 3u) * 8));
        return P::masked(u, m);
    }
    // a high bit for each active column of any piece
    __device__ __forceinline__ void active(int32_t p, uint32_t (&m)[kVec / 4]) const {
        const int32_t at = column(p);
#pragma unroll
        for (int j = 0; j < kVec / 4; ++j) {
            uint8_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = mask[min(max(at + j * 4 + i, 0), n - 1)];
            m[j] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (at + j * 4 + i >= 0 && at + j * 4 + i < n && b[i]) m[j] |= 0x80u << (8 * i);
        }
    }
    template <bool kMask>
    __device__ __forceinline__ uint4 keep_active(uint4 u, int32_t p) const {
        if constexpr (kMask) {
            if (interior(p)) {
                MaskWords w;
                load_mask(p, w);
                return masked(u, w);
            }
            uint32_t m[kVec / 4];
            active(p, m);
            u = P::masked(u, m);
        }
        return u;
    }
    // piece p with minus infinity in inactive columns
    template <bool kMask>
    __device__ __forceinline__ uint4 get(int32_t p) const { return keep_active<kMask>(load(p), p); }
    // one column as a key of the order of the strongest
    template <bool kMask>
    __device__ __forceinline__ uint64_t key(int32_t c) const;
};

// Running maximum, sum and weighted sum of what a thread (or a group) has seen.
struct Running {
    float m, s, w;

    __device__ __forceinline__ Running() : m(minus_inf()), s(0.f), w(0.f) {}  // nothing yet

    __device__ __forceinline__ float reference() const { return m == minus_inf() ? 0.f : m; }
    // moves the sums to the maximum `to` >= m
    __device__ __forceinline__ void raise(float to, float c) {
        if (m == to) return;
        const float d = max_nan((m - to) * c, kNoExponent), r = exp2_fast(d);
        w = (w + d * s) * r;
        s *= r;
        m = to;
    }
};

// Two sums of a thread side by side (packed arithmetic).
struct Pairwise {
    float2 s = make_float2(0.f, 0.f), w = make_float2(0.f, 0.f);
};

// Adds a piece's exponentials: a subtraction, a product, a comparison (which
// keeps 0 * infinity out of the weighted sum and lets NaN pass), an
// exponential, a sum and an fma for each element.
template <typename T>
__device__ __forceinline__ void add_piece(Pairwise& r, const uint4& u, float2 minus_ref, float2 c) {
#pragma unroll
    for (int i = 0; i < PieceOf<T>::kVec / 2; ++i) {
        float2 t = mul2(add2(PieceOf<T>::pair(u, i), minus_ref), c);
        t.x = max_nan(t.x, kNoExponent);
        t.y = max_nan(t.y, kNoExponent);
        const float2 e = make_float2(exp2_fast(t.x), exp2_fast(t.y));
        r.s = add2(r.s, e);
        r.w = fma2(e, t, r.w);
    }
}

constexpr int kLogprobsBatch = 4;  // pieces of a thread that are looked at together
constexpr int kTopSlots = 8;       // parts of a thread's share whose maxima are kept

// A thread's share of a row, pieces first, first + step, ..., in batches.
// kTop: the piece that holds the maximum (the first of equal ones) goes to
// *best, and the maxima of up to kTopSlots runs of `slot` batches to slots[i *
// threads]. Loads of one batch are in flight together, and other warps' beside them:
// registers for a second batch cost more warps than they bring.
template <typename T, bool kMask, bool kTop, bool kShort>
__device__ __forceinline__ Running scan_row(const PiecedRow<T>& row, int32_t first, int32_t last, int32_t step, float c, int32_t* best,
                                            float* slots, int32_t slot, int32_t threads) {
    using P = PieceOf<T>;
    Running r;
    Pairwise sums;
    const float2 c2 = make_float2(c, c);
    const uint4 none = make_uint4(P::kMinusInf, P::kMinusInf, P::kMinusInf, P::kMinusInf);
    float slot_max = minus_inf();
    int32_t left = slot;
    for (int32_t p = first; p < last; p += step * kLogprobsBatch) {
        uint4 u[kLogprobsBatch];
        const bool inside = p + 3 * step < last && (kMask ? row.interior(p) && row.interior(p + 3 * step) : row.whole(p) && row.whole(p + 3 * step));
        if (inside && !(kMask && kShort)) {
#pragma unroll
            for (int j = 0; j < kLogprobsBatch; ++j) u[j] = row.load_whole(p + j * step);
            if constexpr (kMask) {  // all loads before the first use
                typename PiecedRow<T>::MaskWords words[kLogprobsBatch];
#pragma unroll
                for (int j = 0; j < kLogprobsBatch; ++j) row.load_mask(p + j * step, words[j]);
#pragma unroll
                for (int j = 0; j < kLogprobsBatch; ++j) u[j] = row.masked(u[j], words[j]);
            }
        } else if constexpr (kMask && kShort) {  // each piece for itself: a row's ends are a good part of its batches
            typename PiecedRow<T>::MaskWords words[kLogprobsBatch];
            bool in[kLogprobsBatch];
#pragma unroll
            for (int j = 0; j < kLogprobsBatch; ++j) {
                in[j] = p + j * step < last && row.interior(p + j * step);
                if (!in[j]) continue;
                u[j] = row.load_whole(p + j * step);
                row.load_mask(p + j * step, words[j]);
            }
#pragma unroll
            for (int j = 0; j < kLogprobsBatch; ++j)
                u[j] = in[j] ? row.masked(u[j], words[j]) : p + j * step < last ? row.template get<true>(p + j * step) : none;
        } else {
#pragma unroll
            for (int j = 0; j < kLogprobsBatch; ++j) u[j] = p + j * step < last ? row.template get<kMask>(p + j * step) : none;
        }
        uint32_t w[kLogprobsBatch];
#pragma unroll
        for (int j = 0; j < kLogprobsBatch; ++j) w[j] = P::max_words(u[j]);
        const float m = P::word_max(P::max_words(P::max_words(w[0], w[1]), P::max_words(w[2], w[3])));
        if (m > r.m) {
            if constexpr (kTop) {
#pragma unroll
                for (int j = kLogprobsBatch - 1; j >= 0; --j)
                    if (P::word_max(w[j]) == m) *best = p + j * step;
            }
            const float d = max_nan((r.m - m) * c, kNoExponent), f = exp2_fast(d);  // as Running::raise
            const float2 f2 = make_float2(f, f);
            sums.w = mul2(fma2(make_float2(d, d), sums.s, sums.w), f2);
            sums.s = mul2(sums.s, f2);
            r.m = m;
        }
        if constexpr (kTop) {
            if (slots) {
                slot_max = fmaxf(slot_max, m);
                if (--left == 0 || p + step * kLogprobsBatch >= last) {
                    *slots = slot_max;
                    slots += threads;
                    slot_max = minus_inf();
                    left = slot;
                }
            }
        }
        const float ref = -r.reference();
        const float2 ref2 = make_float2(ref, ref);
#pragma unroll
        for (int j = 0; j < kLogprobsBatch; ++j) add_piece<T>(sums, u[j], ref2, c2);
    }
    r.s = sums.s.x + sums.s.y;
    r.w = sums.w.x + sums.w.y;
    return r;
}
static_assert(kLogprobsBatch == 4, "the maxima above");

template <int kThreads>
__device__ __forceinline__ Running reduce_warp(Running r, float c) {
    float m = r.m;
#pragma unroll
    for (int o = kThreads / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    r.raise(m, c);
#pragma unroll
    for (int o = kThreads / 2; o; o >>= 1) {
        r.s += __shfl_xor_sync(0xffffffffu, r.s, o);
        r.w += __shfl_xor_sync(0xffffffffu, r.w, o);
    }
    return r;
}

// What a row's outputs need.
struct RowStats {
    float m, l;  // M, L; an empty row: 0 and +infinity
    float h;     // entropy
    __device__ __forceinline__ RowStats(const Running& r) {
        if (r.m == minus_inf() && r.s == 0.f) {
            m = 0.f;
            l = -minus_inf();
            h = 0.f;
        } else {
            m = r.m;
            l = log2f(r.s);
            h = max_nan(kLn2 * (l - r.w / r.s), 0.f);
        }
    }
};

// The log probability of an active column of value x. (Not by way of t_j, which
// overflows earlier.) Minus infinity gives itself, but in a row whose sum is NaN.
__device__ __forceinline__ float value_logprob(float x, const RowStats& st, float scale) { return (x - st.m) * scale - kLn2 * st.l; }

// A target's value. `kind`: 0 an active column, 1 none (-1), 2 not a column, 3 an inactive column.
template <typename T>
__device__ __forceinline__ float target_value(const LogprobsArgs& a, int64_t r, int i, const T* row, const uint8_t* mask, int* kind) {
    const int64_t j = a.targets[r * a.T + i];
    *kind = j >= 0 && j < a.n ? (mask && !mask[j] ? 3 : 0) : j == -1 ? 1 : 2;
    return *kind ? 0.f : to_f32(row[j]);
}
__device__ __forceinline__ void write_target(const LogprobsArgs& a, int64_t r, int i, float x, int kind, const RowStats& st) {
    if (kind == 2) atomicCAS(a.status, 0, kDeviceInput);
    a.logprob[r * a.T + i] = kind == 0 ? value_logprob(x, st, a.scale) : kind == 1 ? 0.f : kind == 3 ? minus_inf() : __uint_as_float(0x7fffffffu);
}

// The target of thread t of the group that holds the row, read before the scan.
struct Ahead {
    float x = 0.f;
    int kind = 1;
    template <typename T>
    __device__ __forceinline__ Ahead(const LogprobsArgs& a, int64_t r, const T* row, const uint8_t* mask, int t) {
        if (t < a.T) x = target_value(a, r, t, row, mask, &kind);
    }
};

// Writes what does not depend on the strongest columns; every thread of the
// group that holds the row calls it (thread t of `threads`).
template <typename T>
__device__ __forceinline__ void write_row(const LogprobsArgs& a, int64_t r, const T* row, const uint8_t* mask, const RowStats& st,
                                          const Ahead& ahead, int t, int threads) {
    if (t == 0) {
        a.entropy[r] = st.h;
        a.stats[2 * r] = st.m;
        a.stats[2 * r + 1] = st.l;
    }
    if (t < a.T) write_target(a, r, t, ahead.x, ahead.kind, st);
    for (int i = t + threads; i < a.T; i += threads) {
        int kind;
        const float x = target_value(a, r, i, row, mask, &kind);
        write_target(a, r, i, x, kind, st);
    }
}

// ---------------------------------------------------------------- the strongest columns

// A column's place in the order of the strongest: larger value, then lower
// index, first. 0: not listed (inactive, minus infinity, NaN).
__device__ __forceinline__ uint64_t rank_key(float v, int32_t column) {
    if (!(v > minus_inf())) return 0;
    uint32_t b = __float_as_uint(v);
    if (b == 0x80000000u) b = 0;  // the zeros are equal
    b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return static_cast<uint64_t>(b) << 32 | (0xffffffffu - static_cast<uint32_t>(column));
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t b = static_cast<uint32_t>(key >> 32);
    return __uint_as_float((b & 0x80000000u) ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ int32_t key_column(uint64_t key) { return static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(key)); }

template <typename T>
template <bool kMask>
__device__ __forceinline__ uint64_t PiecedRow<T>::key(int32_t c) const {
    if (c < 0 || c >= n || (kMask && !mask[c])) return 0;
    return rank_key(to_f32(x[c]), c);
}

__device__ __forceinline__ uint64_t warp_max_key(uint64_t key) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(key >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(key >> 32) == hi ? static_cast<uint32_t>(key) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}

__device__ __forceinline__ void write_top(const LogprobsArgs& a, int64_t r, int i, uint64_t key, const RowStats& st) {
    a.top_idx[r * a.k + i] = key ? key_column(key) : -1;
    a.top_logprob[r * a.k + i] = key ? value_logprob(key_value(key), st, a.scale) : minus_inf();
}

// ---------------------------------------------------------------- short rows: a warp each

// The strongest columns one after another: the largest of the lanes' own
// maxima is next, and its lane's columns below it are searched, by the whole
// warp, for that lane's next maximum.
template <typename T, bool kMask>
__device__ __forceinline__ void warp_top(const LogprobsArgs& a, int64_t r, const PiecedRow<T>& row, float m, int32_t best, const RowStats& st) {
    constexpr int kVec = PieceOf<T>::kVec;
    const int lane = threadIdx.x & 31;
    uint64_t own = 0;
    if (m > minus_inf()) {
#pragma unroll
        for (int j = kVec - 1; j >= 0; --j) own = max(own, row.template key<kMask>(row.column(best) + j));
    }
    uint64_t taken = 0;  // this lane's of the last 32
    const int32_t per = (row.pieces + 31) / 32 * kVec;  // columns of a lane
    for (int i = 0; i < a.k; ++i) {
        const uint64_t key = warp_max_key(own);
        if ((i & 31) == lane) taken = key;
        if (key != 0) {
            const uint32_t from = __ballot_sync(0xffffffffu, own == key);
            const int owner = __ffs(from) - 1;
            uint64_t next = 0;
            for (int32_t e = lane; e < per; e += 32) {
                const uint64_t k = row.template key<kMask>(row.column(owner + e / kVec * 32) + e % kVec);
                if (k < key) next = max(next, k);
            }
            next = warp_max_key(next);
            if (lane == owner) own = next;
        }
        if ((i & 31) == 31 || i + 1 == a.k) {
            const int at = (i & ~31) + lane;
            if (at <= i) write_top(a, r, at, taken, st);
        }
    }
}

// Rows of up to kRankColumns columns: every column's rank is the number of larger keys.
constexpr int kRankColumns = 256;
template <typename T, bool kMask>
__device__ __forceinline__ void warp_rank(const LogprobsArgs& a, int64_t r, const PiecedRow<T>& row, uint64_t* keys, const RowStats& st) {
    const int lane = threadIdx.x & 31, n = row.n, even = (n + 1) & ~1;
    int active = 0;
    for (int j = lane; j < even; j += 32) {
        const uint64_t key = row.template key<kMask>(j);  // 0 behind the end
        keys[j] = key;
        active += key != 0;
    }
    active = __reduce_add_sync(0xffffffffu, active);
    __syncwarp();
    for (int j = lane; j < n; j += 32) {
        const uint64_t mine = keys[j];
        if (mine == 0) continue;
        int rank = 0;
#pragma unroll 4
        for (int i = 0; i < even; i += 2) {
            const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(keys + i);
            rank += (k.x > mine) + (k.y > mine);
        }
        if (rank < a.k) write_top(a, r, rank, mine, st);
    }
    for (int i = active + lane; i < a.k; i += 32) write_top(a, r, i, 0, st);
}

// kTop: 0 none, 1 one after another, 2 by ranks.
template <typename T, bool kMask, int kTop>
__global__ void __launch_bounds__(256) logprobs_warp_kernel(const LogprobsArgs a) {
    __shared__ alignas(16) uint64_t keys[kTop == 2 ? 8 * kRankColumns : 2];
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (r >= a.rows) return;
    const T* x = static_cast<const T*>(a.x) + r * a.ld;
    const uint8_t* mask = kMask ? a.mask + r * a.ld_mask : nullptr;
    const PiecedRow<T> row(x, mask, a.n, x);
    const Ahead ahead(a, r, x, mask, lane);
    int32_t best = 0;
    const Running mine = scan_row<T, kMask, kTop == 1, true>(row, lane, row.pieces, 32, a.c, &best, nullptr, 0, 0);
    const RowStats st(reduce_warp<32>(mine, a.c));
    write_row(a, r, x, mask, st, ahead, lane, 32);
    if constexpr (kTop == 1) warp_top<T, kMask>(a, r, row, mine.m, best, st);
    if constexpr (kTop == 2) warp_rank<T, kMask>(a, r, row, keys + (threadIdx.x >> 5) * kRankColumns, st);
}

// ---------------------------------------------------------------- long rows: a block, or a cluster of blocks

constexpr int kTopBuffer = 512;

template <int kThreads>
struct alignas(16) TopShared {
    uint64_t found[kTopBuffer];
    uint64_t best[kLogprobsMaxTop];
    float slots[kTopSlots * kThreads];  // maxima of the threads' runs of batches
    uint16_t list[kTopSlots * kThreads];
    int32_t listed, count;
    uint64_t bound, bounds[16];
};

// The k largest of found[0 .. count) into best, descending (0 where there are fewer).
template <int kThreads>
__device__ __forceinline__ void rank_found(TopShared<kThreads>* sh, int count, int k) {
    for (int i = threadIdx.x; i < k; i += kThreads) sh->best[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const uint64_t mine = sh->found[i];
        int rank = 0, j = 0;
#pragma unroll 1
        for (; j + 8 <= count; j += 8) {
            ulonglong2 f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = *reinterpret_cast<const ulonglong2*>(sh->found + j + 2 * e);
#pragma unroll
            for (int e = 0; e < 4; ++e) rank += (f[e].x > mine) + (f[e].y > mine);
        }
#pragma unroll 1
        for (; j < count; ++j) rank += sh->found[j] > mine;
        if (rank < k) sh->best[rank] = mine;
    }
    __syncthreads();
}

// The k largest of `lists` descending lists of k keys (0: none) into best. They
// are gathered first: with the lists' common bound hardly more than k are left.
// Where they are too many, a key's rank is its place in its own list and the
// number of larger keys in each other one.
template <int kThreads>
__device__ __forceinline__ void merge_lists(TopShared<kThreads>* sh, const uint64_t* all, int lists, int k) {
    if (threadIdx.x == 0) sh->count = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < lists * k; i += kThreads) {
        if (all[i] == 0) continue;
        const int at = atomicAdd(&sh->count, 1);
        if (at < kTopBuffer) sh->found[at] = all[i];
    }
    __syncthreads();
    const int count = sh->count;
    if (count <= kTopBuffer) {
        rank_found<kThreads>(sh, count, k);
        return;
    }
    for (int i = threadIdx.x; i < lists * k; i += kThreads) {
        const uint64_t mine = all[i];
        if (mine == 0) continue;
        int rank = i % k;
        for (int l = 0; l < lists && rank < k; ++l) {
            if (l == i / k) continue;
            int lo = 0, hi = k;  // the first place whose key is not larger
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (all[l * k + mid] > mine) lo = mid + 1;
                else hi = mid;
            }
            rank += lo;
        }
        if (rank < k) sh->best[rank] = mine;
    }
    __syncthreads();
}

// Bounds that at least k of the threads' keys reach, and hardly more (1 where
// there are fewer keys): thread t's keys are found[0 .. kThreads). One warp
// searches by halves, among the values, and among the columns of one value only
// where many are equal.
template <int kThreads>
__device__ __forceinline__ uint64_t search_bound(const uint64_t* found, int k) {
    constexpr int kPer = kThreads / 32;
    const int most = k + (k >> 2);
    uint64_t mine[kPer];
    uint32_t least = 0xffffffffu, largest = 0;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        mine[i] = found[i * 32 + (threadIdx.x & 31)];
        const uint32_t v = static_cast<uint32_t>(mine[i] >> 32);
        n += v != 0;
        largest = max(largest, v);
        if (v) least = min(least, v);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (n < k) return 1;
    uint32_t lo = __reduce_min_sync(0xffffffffu, least), hi = __reduce_max_sync(0xffffffffu, largest);
    while (lo < hi && n > most) {
        const uint32_t mid = lo + ((hi - lo) >> 1) + 1;
        int count = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) count += static_cast<uint32_t>(mine[i] >> 32) >= mid;
        count = __reduce_add_sync(0xffffffffu, count);
        if (count >= k) {
            lo = mid;
            n = count;
        } else {
            hi = mid - 1;
        }
    }
    uint64_t bound = static_cast<uint64_t>(lo) << 32;
    if (n <= most) return bound;
    uint32_t low = 0, high = 0xffffffffu;  // lo is the k-th value: columns decide
    while (low < high && n > most) {
        const uint32_t mid = low + ((high - low) >> 1) + 1;
        int count = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) count += mine[i] >= (bound | mid);
        count = __reduce_add_sync(0xffffffffu, count);
        if (count >= k) {
            low = mid;
            n = count;
        } else {
            high = mid - 1;
        }
    }
    return bound | low;
}

// The k strongest columns of pieces [first, last), which this block's threads
// have seen with their stride. At least k threads' maxima reach the bound; only the
// runs of batches whose maximum does are read again. Ties and rows whose large
// columns all fall to few threads give more candidates than the buffer takes:
// the k-th best of those found is then a higher bound.
template <typename T, bool kMask, int kThreads>
__device__ __noinline__ void block_top(TopShared<kThreads>* sh, const PiecedRow<T>& row, int32_t first, int32_t last, int32_t slot,
                                       float m, int32_t best, int k, int blocks) {
    constexpr int kVec = PieceOf<T>::kVec;
    const int32_t per = slot * kLogprobsBatch;  // pieces of a run
    // at most this key
    auto upper = [&](float v, int32_t piece) { return v > minus_inf() ? rank_key(v, max(row.column(piece), 0)) : 0; };
    const uint64_t lower = m > minus_inf() ? rank_key(m, row.column(best) + kVec - 1) : 0;
    sh->found[threadIdx.x] = lower;
    if (threadIdx.x == 0) sh->listed = sh->count = 0;
    __syncthreads();
    uint64_t bound = 1;
    if (blocks > 1) {
        // Every block has ceil(k / blocks) columns that reach its own bound for so
        // many, so k of the row's reach the least of these.
        if (threadIdx.x < 32) {
            bound = search_bound<kThreads>(sh->found, (k + blocks - 1) / blocks);
            if (threadIdx.x < blocks) {
                const uint32_t at = map_shared_rank(smem_u32(&sh->bounds[cluster_ctarank()]), threadIdx.x);
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(bound) : "memory");
            }
        }
        cluster_sync_all();
        bound = sh->bounds[0];
        for (int i = 1; i < blocks; ++i) bound = min(bound, sh->bounds[i]);
    }
    if (bound <= 1) {
        if (threadIdx.x < 32) {
            bound = search_bound<kThreads>(sh->found, k);
            if (threadIdx.x == 0) sh->bound = bound;
        }
        __syncthreads();
        bound = sh->bound;
    }
    for (;;) {
        const float value = bound > 1 ? key_value(bound) : minus_inf();  // what is below is below the bound
        if (m >= value && upper(m, best) >= bound) {
#pragma unroll 1
            for (int i = 0; i < kTopSlots; ++i) {
                const int32_t p = first + threadIdx.x + i * per * kThreads;
                if (p >= last) break;
                const float v = sh->slots[i * kThreads + threadIdx.x];
                if (v >= value && upper(v, p) >= bound) sh->list[atomicAdd(&sh->listed, 1)] = static_cast<uint16_t>(i * kThreads + threadIdx.x);
            }
        }
        __syncthreads();
        const int32_t total = per * sh->listed;
#pragma unroll 2
        for (int32_t i = threadIdx.x; i < total; i += kThreads) {
            const int32_t e = sh->list[i / per], p = first + e % kThreads + (e / kThreads * per + i % per) * kThreads;
            if (p >= last) continue;
            const uint4 u = row.template get<kMask>(p);
            uint32_t reach = 0;
#pragma unroll
            for (int j = 0; j < kVec / 2; ++j) {
                const float2 v = PieceOf<T>::pair(u, j);
                reach |= (v.x >= value ? 1u : 0u) << (2 * j) | (v.y >= value ? 2u : 0u) << (2 * j);
            }
            for (; reach; reach &= reach - 1) {
                const uint64_t key = row.template key<kMask>(row.column(p) + __ffs(reach) - 1);
                if (key < bound) continue;
                const int to = atomicAdd(&sh->count, 1);
                if (to < kTopBuffer) sh->found[to] = key;
            }
        }
        __syncthreads();
        const int count = sh->count;
        rank_found<kThreads>(sh, min(count, kTopBuffer), k);
        if (count <= kTopBuffer) break;
        bound = sh->best[k - 1];
        if (threadIdx.x == 0) sh->listed = sh->count = 0;
        __syncthreads();
    }
}

// kThreads threads of each of a cluster's blocks share a row. 56 registers, nine
// blocks of 128 threads an SM: 4096 x 131072 bf16 in 155 us, 6.9 TB/s (with eight 167).
template <typename T, bool kMask, bool kTop, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 128 ? 9 : 4) logprobs_block_kernel(const LogprobsArgs a, int blocks) {
    __shared__ float part[kThreads / 32][3];
    __shared__ float gathered[16][3];
    extern __shared__ uint64_t all_best[];  // kTop, blocks > 1: [blocks, k]
    __shared__ TopShared<kThreads> top;  // kTop
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = blocks > 1 ? cluster_ctarank() : 0;
    if (blocks > 1) cluster_sync_all();  // every block has started before its shared memory is written
    const int64_t r = blockIdx.x / blocks;
    const T* x = static_cast<const T*>(a.x) + r * a.ld;
    const uint8_t* mask = kMask ? a.mask + r * a.ld_mask : nullptr;
    const PiecedRow<T> row(x, mask, a.n, x);
    const Ahead ahead(a, r, x, mask, rank == 0 ? threadIdx.x : a.T);
    const int32_t share = (row.pieces + blocks - 1) / blocks;
    const int32_t p0 = min(row.pieces, static_cast<int32_t>(rank) * share), p1 = min(row.pieces, p0 + share);
    int32_t best = 0;
    const int32_t per_thread = (share + kThreads * kLogprobsBatch - 1) / (kThreads * kLogprobsBatch);  // batches
    const int32_t slot = max(1, (per_thread + kTopSlots - 1) / kTopSlots);
    const Running mine = scan_row<T, kMask, kTop, false>(row, p0 + threadIdx.x, p1, kThreads, a.c, &best, kTop ? top.slots + threadIdx.x : nullptr,
                                                  slot, kThreads);
    const Running sum = reduce_warp<32>(mine, a.c);
    if (lane == 0) {
        part[warp][0] = sum.m;
        part[warp][1] = sum.s;
        part[warp][2] = sum.w;
    }
    __syncthreads();
    Running all;
    if (lane < kThreads / 32) {
        all.m = part[lane][0];
        all.s = part[lane][1];
        all.w = part[lane][2];
    }
    all = reduce_warp<32>(all, a.c);
    if constexpr (kTop) block_top<T, kMask, kThreads>(&top, row, p0, p1, slot, mine.m, best, a.k, blocks);
    if (blocks > 1) {
        // every block's sums and strongest columns to the first block's shared memory
        if (threadIdx.x == 0) {
            const uint32_t at = map_shared_rank(smem_u32(&gathered[rank][0]), 0);
            asm volatile("st.shared::cluster.f32 [%0], %1;\n\tst.shared::cluster.f32 [%0+4], %2;\n\tst.shared::cluster.f32 [%0+8], %3;" ::"r"(at),
                         "f"(all.m), "f"(all.s), "f"(all.w) : "memory");
        }
        if constexpr (kTop) {
            for (int i = threadIdx.x; i < a.k; i += kThreads) {
                const uint32_t at = map_shared_rank(smem_u32(&all_best[rank * a.k + i]), 0);
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(top.best[i]) : "memory");
            }
        }
        cluster_sync_all();
        if (rank != 0) return;
        all = Running();
        if (lane < blocks) {
            all.m = gathered[lane][0];
            all.s = gathered[lane][1];
            all.w = gathered[lane][2];
        }
        all = reduce_warp<32>(all, a.c);
        if constexpr (kTop) {
            merge_lists<kThreads>(&top, all_best, blocks, a.k);
        }
    }
    const RowStats st(all);
    write_row(a, r, x, mask, st, ahead, threadIdx.x, kThreads);
    if constexpr (kTop)
        for (int i = threadIdx.x; i < a.k; i += kThreads) write_top(a, r, i, top.best[i], st);
}

// ---------------------------------------------------------------- gradient

struct LogprobsBwdArgs {
    const void* x;
    const int64_t* targets;
    const uint8_t* mask;
    int64_t rows, n, ld, ld_mask, ld_dx;
    int32_t T, k;
    float scale, c;
    const float* stats;
    const float* entropy;
    const float* g_logprob;   // [rows, T] or NULL
    const float* g_entropy;   // [rows] or NULL
    const int32_t* top_idx;   // [rows, k] with g_top
    const float* g_top;       // [rows, k] or NULL
    void* dx;
    int* status;
};

// The i-th of a row's T + k columns with a gradient of their own: its column
// (-1: none) and gradient.
template <typename T>
__device__ __forceinline__ int32_t given_column(const LogprobsBwdArgs& a, int64_t r, int i, const T* x, const uint8_t* mask, float m, float* g) {
    int64_t j;
    if (i < a.T) {
        j = a.g_logprob ? a.targets[r * a.T + i] : -1;
        *g = j >= 0 ? a.g_logprob[r * a.T + i] : 0.f;
    } else {
        j = a.top_idx[r * a.k + i - a.T];
        *g = j >= 0 ? a.g_top[r * a.k + i - a.T] : 0.f;
    }
    if (j < -1 || j >= a.n) {
        atomicCAS(a.status, 0, kDeviceInput);
        j = -1;
    }
    // a column of probability zero passes no gradient
    if (j >= 0 && ((mask && !mask[j]) || (to_f32(x[j]) - m) * a.scale == minus_inf())) j = -1;
    if (j < 0) *g = 0.f;
    return static_cast<int32_t>(j);
}

// dx_j = scale * (sum of what was given to j) + p_j * (A + B * log2 p_j),
// log2 p_j = t_j - L, A = -scale * (G + g_entropy * entropy),
// B = -scale * g_entropy * ln 2, G = the sum of all that was given.

// Pieces of a lane in flight, and blocks of 256 threads an SM holds at least.
// Registers decide. Plain rows have the next pieces in flight while some are worked
// on (4096 x 131072 bf16 by pieces and blocks: 4, 3: 370 us; 3, 4: 324; 2, 5: 325).
// Masked rows and rows of another phase load a batch at a time (8192 x 32768 bf16 with a
// mask for each row: 4, 4: 223 us; 2, 5: 234; 3, 4: 215; 4, 3: 225).
struct BwdCfg {
    static constexpr int kPieces = 3, kBlocks = 4;
};

// Calls f(column, gradient) in every lane for the given columns from c0 to c1,
// in their order. Lane i holds the i-th of the first 32 (j, g); later ones are
// read again, for every piece, and decide from there on (4096 x 131072 bf16, given
// and listed columns together: 1 316 us, 32 325, 33 440, 65 627, 256 2,112).
template <typename T, typename F>
__device__ __forceinline__ void each_given(const LogprobsBwdArgs& a, int64_t r, const T* x, const uint8_t* mask, float m, int given, int32_t j,
                                           float g, int32_t c0, int32_t c1, F&& f) {
    for (int b = 0; b < given; b += 32) {
        if (b > 0) j = b + static_cast<int>(threadIdx.x & 31) < given ? given_column(a, r, b + (threadIdx.x & 31), x, mask, m, &g) : -1;
        for (uint32_t left = __ballot_sync(0xffffffffu, j >= c0 && j < c1); left; left &= left - 1) {
            const int from = __ffs(left) - 1;
            f(__shfl_sync(0xffffffffu, j, from), __shfl_sync(0xffffffffu, g, from));
        }
    }
}

// A warp per (row, run of `run` pieces): no warp waits for another. The given
// columns' own gradients are added to the elements before they are rounded.
// Pieces are those of dx, so that stores are whole; kShift: x's rows have
// another phase, and its pieces are joined from the two aligned ones that hold
// them. Bound by HBM (4096 x 131072 bf16 317 us, 6.8 TB/s) but for masked rows of
// another phase, which wait for their loads (43 % of the warps an SM may hold), 40 bytes
// spilled in 16-bit types (999 x 32003 f16: 43 us, 37 % of HBM's rate).
template <typename T, bool kMask, bool kShift>
__global__ void __launch_bounds__(256, BwdCfg::kBlocks) logprobs_bwd_kernel(const LogprobsBwdArgs a, int32_t run, int64_t runs, int64_t items) {
    using P = PieceOf<T>;
    constexpr int kVec = P::kVec, kBwdPieces = BwdCfg::kPieces;
    constexpr bool kPlain = !kMask && !kShift;
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (item >= items) return;
    const int64_t r = item / runs;
    const T* x = static_cast<const T*>(a.x) + r * a.ld;
    T* dx = static_cast<T*>(a.dx) + r * a.ld_dx;
    const uint8_t* mask = kMask ? a.mask + r * a.ld_mask : nullptr;
    const PiecedRow<T> row(x, mask, a.n, dx);
    const int32_t first = static_cast<int32_t>(item - r * runs) * run, last = min(row.pieces, first + run);
    const float2 m = *reinterpret_cast<const float2*>(a.stats + 2 * r);
    const int given = a.T + (a.g_top ? a.k : 0);
    // the first 32 given columns, one a lane; all of their gradients' sum
    float g = 0.f, sum = 0.f;
    int32_t j = -1;
    if (lane < given) j = given_column(a, r, lane, x, mask, m.x, &g);
    sum = g;
    for (int i = lane + 32; i < given; i += 32) {
        float more;
        given_column(a, r, i, x, mask, m.x, &more);
        sum += more;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float gh = a.g_entropy ? a.g_entropy[r] : 0.f;
    float A = -a.scale * __fmaf_rn(gh, gh != 0.f ? a.entropy[r] : 0.f, sum), B = -a.scale * gh * kLn2;
    if (m.y == -minus_inf()) A = B = 0.f;  // an empty row passes no gradient, whatever it is given
    const float2 ref = make_float2(-m.x, -m.x), c2 = make_float2(a.c, a.c), l2 = make_float2(-m.y, -m.y);
    const float2 A2 = make_float2(A, A), B2 = make_float2(B, B);
    // a row of NaN, or given gradients that are not finite: p * (A + B * log2 p) is NaN for p = 0 too, inactive columns are 0 all the same
    const bool broken = !(m.x == m.x && m.y == m.y && fabsf(A) <= kLargest && fabsf(B) * -kNoExponent <= kLargest);
    // whole pieces
    const int32_t w0 = max(first, row.skip ? 1 : 0), w1 = min(last, (row.n + row.skip) / kVec);
    const uint4 none = make_uint4(P::kMinusInf, P::kMinusInf, P::kMinusInf, P::kMinusInf);
    uint4 next[kPlain ? kBwdPieces : 1];
    auto fetch = [&](int32_t p0) {
#pragma unroll
        for (int i = 0; i < kBwdPieces; ++i) {
            const int32_t p = p0 + i * 32 + lane;
            next[kPlain ? i : 0] = p < w1 ? row.load_whole(p) : none;
        }
    };
    if constexpr (kPlain) fetch(w0);
    for (int32_t p0 = w0; p0 < w1; p0 += 32 * kBwdPieces) {
        uint4 u[kBwdPieces];
        if constexpr (kPlain) {
#pragma unroll
            for (int i = 0; i < kBwdPieces; ++i) u[i] = next[i];
            fetch(p0 + 32 * kBwdPieces);
        } else {  // all loads before the first use
            uint4 hi[kShift ? kBwdPieces : 1];
            typename PiecedRow<T>::MaskWords words[kMask ? kBwdPieces : 1];
            bool in[kBwdPieces];
#pragma unroll
            for (int i = 0; i < kBwdPieces; ++i) {
                const int32_t p = p0 + i * 32 + lane;
                in[i] = p < w1 && row.interior(p);
                if (!in[i]) continue;
                if constexpr (kShift) row.load_around(p, u[i], hi[i]);
                else u[i] = row.load_whole(p);
                if constexpr (kMask) row.load_mask(p, words[i]);
            }
#pragma unroll
            for (int i = 0; i < kBwdPieces; ++i) {
                const int32_t p = p0 + i * 32 + lane;
                if (in[i]) {
                    if constexpr (kShift) u[i] = row.shifted(u[i], hi[i]);
                    if constexpr (kMask) u[i] = row.masked(u[i], words[i]);
                } else {
                    u[i] = p < w1 ? row.template get<kMask>(p) : none;
                }
            }
        }
        // exponents of minus infinity, as in add_piece
        uint32_t least = P::min_words(u[0]);
#pragma unroll
        for (int i = 1; i < kBwdPieces; ++i) least = P::min_words(least, P::min_words(u[i]));
        const bool low = !((P::word_min(least) + ref.x) * a.c > kLowExponent) || !(m.y < 1e30f);
        const int32_t c0 = row.column(p0), c1 = c0 + 32 * kBwdPieces * kVec;
        const uint32_t here = __ballot_sync(0xffffffffu, j >= c0 && j < c1);
#pragma unroll
        for (int i = 0; i < kBwdPieces; ++i) {
            if (p0 + i * 32 >= w1) break;
            const int32_t p = p0 + i * 32 + lane, at = row.column(p);
            float2 d[kVec / 2];
#pragma unroll
            for (int e = 0; e < kVec / 2; ++e) {
                // log2 p, p, p * (A + B log2 p)
                float2 t = fma2(add2(P::pair(u[i], e), ref), c2, l2);
                if (low) {
                    t.x = max_nan(t.x, kNoExponent);
                    t.y = max_nan(t.y, kNoExponent);
                }
                d[e] = mul2(make_float2(exp2_fast(t.x), exp2_fast(t.y)), fma2(t, B2, A2));
            }
            if (kMask && broken && p < w1) {
                uint32_t act[kVec / 4];
                row.active(p, act);
#pragma unroll
                for (int e = 0; e < kVec / 2; ++e) {
                    const uint32_t b = act[2 * e / 4] >> (2 * e % 4 * 8);
                    if (!(b & 0x80u)) d[e].x = 0.f;
                    if (!(b & 0x8000u)) d[e].y = 0.f;
                }
            }
            if (here || given > 32) {
                each_given(a, r, x, mask, m.x, given, j, g, c0, c1, [&](int32_t column, float v) {
#pragma unroll
                    for (int e = 0; e < kVec / 2; ++e) {
                        if (column - at == 2 * e) d[e].x = __fmaf_rn(a.scale, v, d[e].x);
                        if (column - at == 2 * e + 1) d[e].y = __fmaf_rn(a.scale, v, d[e].y);
                    }
                });
            }
            if (p >= w1) continue;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < kVec / 2; ++e) {
                if constexpr (sizeof(T) == 4) {
                    w[2 * e] = __float_as_uint(d[e].x);
                    w[2 * e + 1] = __float_as_uint(d[e].y);
                } else {
                    w[e] = pack2<T>(d[e].x, d[e].y);
                }
            }
            *reinterpret_cast<uint4*>(dx + at) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    // the row's ends: an element a lane, those in front of the first whole piece and those behind the last one
    const bool head = first == 0 && row.skip, tail = last == row.pieces && (row.n + row.skip) % kVec != 0;
    if (head || tail) {
        const int32_t w_first = row.column(row.skip ? 1 : 0), w_end = row.column((row.n + row.skip) / kVec);
        int32_t column = -1;
        if (head && lane < kVec && lane < min(w_first, row.n)) column = lane;
        if (tail && lane >= kVec && lane < 2 * kVec && max(w_end, 0) + lane - kVec < row.n && (w_end >= w_first || !head))
            column = max(w_end, 0) + lane - kVec;
        float d = 0.f;
        const bool on = column >= 0 && !(kMask && !mask[column]);
        if (on) {
            const float t = max_nan(__fmaf_rn(to_f32(x[column]) - m.x, a.c, -m.y), kNoExponent);
            d = exp2_fast(t) * __fmaf_rn(t, B, A);
        }
        each_given(a, r, x, mask, m.x, given, j, g, 0, row.n, [&](int32_t c, float v) {
            if (c == column) d = __fmaf_rn(a.scale, v, d);
        });
        if (column >= 0) dx[column] = from_f32<T>(d);
    }
}

}  // namespace maxsim
