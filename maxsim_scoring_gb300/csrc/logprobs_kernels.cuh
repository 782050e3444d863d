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
__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xff800000u); }

// kVec elements (16 bytes) of a row.
template <typename T>
struct Piece {
    static constexpr int kVec = 16 / static_cast<int>(sizeof(T));
    float v[kVec];
    __device__ __forceinline__ void set(uint4 u) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[i] = __uint_as_float(w[i]);
            } else {
                const uint32_t h = (i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu;
                if constexpr (std::is_same_v<T, __half>) v[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
                else v[i] = __uint_as_float(h << 16);
            }
        }
    }
};

// A row seen as aligned 16-byte pieces: piece p holds columns p * kVec - skip
// and on; the first and the last one may reach over the row's ends, and are
// read element by element then.
template <typename T>
struct PiecedRow {
    static constexpr int kVec = Piece<T>::kVec;
    const T* x;
    const uint8_t* mask;
    int64_t n;
    int32_t skip;
    int32_t pieces;

    __device__ __forceinline__ PiecedRow(const T* row, const uint8_t* m, int64_t cols) : x(row), mask(m), n(cols) {
        skip = static_cast<int32_t>(reinterpret_cast<uintptr_t>(row) / sizeof(T)) & (kVec - 1);
        pieces = static_cast<int32_t>((n + skip + kVec - 1) / kVec);
    }
    __device__ __forceinline__ int64_t column(int32_t p) const { return static_cast<int64_t>(p) * kVec - skip; }
    __device__ __forceinline__ bool whole(int32_t p) const { return column(p) >= 0 && column(p) + kVec <= n; }
    // 16 bytes of piece p; what is not the row's is minus infinity
    __device__ __forceinline__ uint4 load(int32_t p) const {
        const int64_t at = column(p);
        if (at >= 0 && at + kVec <= n) return __ldg(reinterpret_cast<const uint4*>(x + at));
        alignas(16) T e[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) e[i] = at + i >= 0 && at + i < n ? x[at + i] : from_f32<T>(minus_inf());
        return *reinterpret_cast<const uint4*>(e);
    }
    // bit i: column i of piece p is active
    __device__ __forceinline__ uint32_t active(int32_t p) const {
        const int64_t at = column(p);
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (at + i >= 0 && at + i < n && mask[at + i]) bits |= 1u << i;
        return bits;
    }
    template <bool kMask>
    __device__ __forceinline__ void get(Piece<T>& e, uint4 u, uint32_t bits) const {
        e.set(u);
        if constexpr (kMask) {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (!(bits >> i & 1)) e.v[i] = minus_inf();
        }
    }
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

template <typename T>
__device__ __forceinline__ float piece_max(const Piece<T>& e) {
    float m = e.v[0];
#pragma unroll
    for (int i = 1; i + 1 < Piece<T>::kVec; i += 2) m = fmax3(m, e.v[i], e.v[i + 1]);
    return fmaxf(m, e.v[Piece<T>::kVec - 1]);
}

template <typename T>
__device__ __forceinline__ void add_piece(Running& r, const Piece<T>& e, float ref, float c) {
#pragma unroll
    for (int i = 0; i < Piece<T>::kVec; ++i) {
        const float t = max_nan((e.v[i] - ref) * c, kNoExponent), y = exp2_fast(t);
        r.s += y;
        r.w = __fmaf_rn(y, t, r.w);
    }
}

constexpr int kLogprobsBatch = 4;  // pieces of a thread in flight

// A thread's share of a row: pieces first, first + step, ... The column of the
// piece that holds the maximum (the first of equal ones) goes to *best.
template <typename T, bool kMask, bool kBest>
__device__ __forceinline__ Running scan_row(const PiecedRow<T>& row, int32_t first, int32_t last, int32_t step, float c, int32_t* best) {
    Running r;
    for (int32_t p = first; p < last; p += step * kLogprobsBatch) {
        uint4 u[kLogprobsBatch];
        uint32_t bits[kLogprobsBatch];
#pragma unroll
        for (int j = 0; j < kLogprobsBatch; ++j)
            if (p + j * step < last) {
                u[j] = row.load(p + j * step);
                if constexpr (kMask) bits[j] = row.active(p + j * step);
            }
#pragma unroll
        for (int j = 0; j < kLogprobsBatch; ++j) {
            if (p + j * step >= last) break;
            Piece<T> e;
            row.template get<kMask>(e, u[j], kMask ? bits[j] : 0u);
            const float m = piece_max(e);
            if (m > r.m) {
                r.raise(m, c);
                if constexpr (kBest) *best = p + j * step;
            }
            add_piece(r, e, r.reference(), c);
        }
    }
    return r;
}

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

// The log probability of one column: minus infinity where it is not active. (Not by way of t_j, which overflows earlier.)
template <typename T>
__device__ __forceinline__ float column_logprob(const T* row, const uint8_t* mask, int64_t j, const RowStats& st, float scale) {
    if (mask && !mask[j]) return minus_inf();
    const float x = to_f32(row[j]);
    if (x == minus_inf()) return x;
    return (x - st.m) * scale - kLn2 * st.l;
}

// Writes what does not depend on the strongest columns; every thread of the
// group that holds the row calls it (thread t of `threads`).
template <typename T>
__device__ __forceinline__ void write_row(const LogprobsArgs& a, int64_t r, const T* row, const uint8_t* mask, const RowStats& st,
                                          int t, int threads) {
    if (t == 0) {
        a.entropy[r] = st.h;
        a.stats[2 * r] = st.m;
        a.stats[2 * r + 1] = st.l;
    }
    for (int i = t; i < a.T; i += threads) {
        const int64_t j = a.targets[r * a.T + i];
        float v = 0.f;
        if (j >= 0 && j < a.n) {
            v = column_logprob(row, mask, j, st, a.scale);
        } else if (j != -1) {
            atomicCAS(a.status, 0, kDeviceInput);
            v = __uint_as_float(0x7fffffffu);
        }
        a.logprob[r * a.T + i] = v;
    }
}

// ---------------------------------------------------------------- short rows: a warp each

template <typename T, bool kMask>
__global__ void __launch_bounds__(256) logprobs_warp_kernel(const LogprobsArgs a) {
    const int lane = threadIdx.x & 31;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); r < a.rows; r += static_cast<int64_t>(gridDim.x) * 8) {
        const T* x = static_cast<const T*>(a.x) + r * a.ld;
        const uint8_t* mask = kMask ? a.mask + r * a.ld_mask : nullptr;
        const PiecedRow<T> row(x, mask, a.n);
        const RowStats st(reduce_warp<32>(scan_row<T, kMask, false>(row, lane, row.pieces, 32, a.c, nullptr), a.c));
        write_row(a, r, x, mask, st, lane, 32);
    }
}

// ---------------------------------------------------------------- long rows: a block, or a cluster of blocks

// A column's place in the order of the strongest: larger value, then lower
// index, first. 0: not listed (inactive, minus infinity, NaN).
__device__ __forceinline__ uint64_t rank_key(float v, int32_t column) {
    if (!(v > minus_inf())) return 0;
    uint32_t b = __float_as_uint(v);
    if (b == 0x80000000u) b = 0;  // the zeros are equal
    b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return static_cast<uint64_t>(b) << 32 | (0xffffffffu - static_cast<uint32_t>(column));
}
__device__ __forceinline__ int32_t key_column(uint64_t key) { return static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(key)); }

constexpr int kTopBuffer = 1024;

struct TopShared {
    uint64_t found[kTopBuffer];
    uint64_t best[kLogprobsMaxTop];
    int32_t list[1024];
    int32_t listed, count;
    uint64_t bound;
};

// The k largest of found[0 .. count) into best, descending (0 where there are fewer).
template <int kThreads>
__device__ __forceinline__ void rank_found(TopShared* sh, int count, int k) {
    for (int i = threadIdx.x; i < k; i += kThreads) sh->best[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const uint64_t mine = sh->found[i];
        int rank = 0;
        for (int j = 0; j < count; ++j) rank += sh->found[j] > mine;
        if (rank < k) sh->best[rank] = mine;
    }
    __syncthreads();
}

// The k strongest columns of pieces [0, last) with this block's stride.
// A thread's own maximum says whether it can hold any of them: at least k
// threads' maxima reach the bound that is searched for here, and only the
// pieces of threads whose maximum reaches it are read again. Ties and rows
// whose large columns all fall to one thread give more candidates than the
// buffer takes: the k-th best of those found is then a higher bound.
template <typename T, bool kMask, int kThreads>
__device__ __forceinline__ void block_top(TopShared* sh, const PiecedRow<T>& row, int32_t first, int32_t last, int32_t step, float m,
                                          int32_t best, int k) {
    constexpr int kVec = Piece<T>::kVec;
    // upper and lower end of what the maximum's piece holds
    const uint64_t upper = m > minus_inf() ? rank_key(m, static_cast<int32_t>(max(row.column(best), static_cast<int64_t>(0)))) : 0;
    const uint64_t lower = m > minus_inf() ? rank_key(m, static_cast<int32_t>(row.column(best) + kVec - 1)) : 0;
    uint64_t lo = 1, hi = ~0ull;
    if (__syncthreads_count(lower != 0) >= k) {
        // the largest bound (or one reached by at most 2 k threads) that k threads reach
        while (lo < hi) {
            const uint64_t mid = lo + ((hi - lo) >> 1) + 1;
            const int n = __syncthreads_count(lower >= mid);
            if (n >= k) lo = mid;
            else hi = mid - 1;
            if (n >= k && n <= 2 * k) break;
        }
    }
    uint64_t bound = lo;
    for (;;) {
        if (threadIdx.x == 0) sh->listed = sh->count = 0;
        __syncthreads();
        if (upper >= bound) sh->list[atomicAdd(&sh->listed, 1)] = threadIdx.x;
        __syncthreads();
        const int32_t per = (last - first + step - 1) / step, total = per * sh->listed;
        for (int32_t i = threadIdx.x; i < total; i += kThreads) {
            const int32_t p = first + sh->list[i / per] + (i % per) * step;
            if (p >= last) continue;
            Piece<T> e;
            row.template get<kMask>(e, row.load(p), kMask ? row.active(p) : 0u);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const uint64_t key = rank_key(e.v[j], static_cast<int32_t>(row.column(p) + j));
                if (key >= bound) {
                    const int at = atomicAdd(&sh->count, 1);
                    if (at < kTopBuffer) sh->found[at] = key;
                }
            }
        }
        __syncthreads();
        const int count = sh->count;
        rank_found<kThreads>(sh, min(count, kTopBuffer), k);
        if (count <= kTopBuffer) break;
        bound = sh->best[k - 1];
        __syncthreads();
    }
}

// kThreads threads of each of a cluster's blocks share a row.
template <typename T, bool kMask, bool kTop, int kThreads>
__global__ void __launch_bounds__(kThreads) logprobs_block_kernel(const LogprobsArgs a, int blocks) {
    __shared__ float part[32][3];
    __shared__ float gathered[16][3];
    __shared__ uint64_t all_best[kTop ? 16 * kLogprobsMaxTop : 1];
    __shared__ TopShared top;  // kTop
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = blocks > 1 ? cluster_ctarank() : 0;
    if (blocks > 1) cluster_sync_all();  // every block has started before its shared memory is written
    for (int64_t r = blockIdx.x / blocks; r < a.rows; r += gridDim.x / blocks) {
        const T* x = static_cast<const T*>(a.x) + r * a.ld;
        const uint8_t* mask = kMask ? a.mask + r * a.ld_mask : nullptr;
        const PiecedRow<T> row(x, mask, a.n);
        const int32_t share = (row.pieces + blocks - 1) / blocks;
        const int32_t p0 = min(row.pieces, static_cast<int32_t>(rank) * share), p1 = min(row.pieces, p0 + share);
        int32_t best = 0;
        Running mine = scan_row<T, kMask, kTop>(row, p0 + threadIdx.x, p1, kThreads, a.c, &best);
        Running sum = reduce_warp<32>(mine, a.c);
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
        if constexpr (kTop) block_top<T, kMask, kThreads>(&top, row, p0, p1, kThreads, mine.m, best, a.k);
        if (blocks > 1) {
            // every block's sums and strongest columns to all blocks' shared memory
            for (uint32_t to = threadIdx.x; to < static_cast<uint32_t>(blocks); to += kThreads) {
                const uint32_t at = map_shared_rank(smem_u32(&gathered[rank][0]), to);
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
            Running g;
            if (lane < blocks) {
                g.m = gathered[lane][0];
                g.s = gathered[lane][1];
                g.w = gathered[lane][2];
            }
            all = reduce_warp<32>(g, a.c);
        }
        const RowStats st(all);
        if (rank == 0) {
            write_row(a, r, x, mask, st, threadIdx.x, kThreads);
            if constexpr (kTop) {
                if (blocks > 1) {
                    for (int i = threadIdx.x; i < blocks * a.k; i += kThreads) top.found[i] = all_best[i];
                    __syncthreads();
                    // keys of 0 rank last
                    rank_found<kThreads>(&top, blocks * a.k, a.k);
                }
                for (int i = threadIdx.x; i < a.k; i += kThreads) {
                    const uint64_t key = top.best[i];
                    a.top_idx[r * a.k + i] = key ? key_column(key) : -1;
                    a.top_logprob[r * a.k + i] = key ? column_logprob(x, mask, key_column(key), st, a.scale) : minus_inf();
                }
            }
        }
        if (blocks > 1) cluster_sync_all();
        else __syncthreads();
    }
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
__device__ __forceinline__ int64_t given_column(const LogprobsBwdArgs& a, int64_t r, int i, const T* x, const uint8_t* mask, float m, float* g) {
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
    return j;
}

// dx_j = scale * (sum of what was given to j) + p_j * (A + B * u_j),
// u_j = t_j - L (log2 p_j), A = -scale * (G + g_entropy * entropy),
// B = -scale * g_entropy * ln 2, G = the sum of all that was given.
struct GradRow {
    float m, l, A, B;
    __device__ __forceinline__ float log2_p(float x, float c) const { return max_nan((x - m) * c - l, kNoExponent); }
    __device__ __forceinline__ float dx(float x, float c) const {
        const float u = log2_p(x, c);
        return exp2_fast(u) * __fmaf_rn(u, B, A);
    }
};

// kGroup threads take kPieces pieces each of one row's run; one group per
// (row, run). No sums but those of the T + k given columns, which every run's
// group adds up again. Bound by HBM.
template <typename T, bool kMask, int kGroup, int kPieces>
__global__ void __launch_bounds__(256) logprobs_bwd_kernel(const LogprobsBwdArgs a, int64_t runs, int64_t items) {
    constexpr int kVec = Piece<T>::kVec;
    const int t = threadIdx.x % kGroup;
    __shared__ float sum_of[8];
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * (256 / kGroup) + threadIdx.x / kGroup; item < items;
         item += static_cast<int64_t>(gridDim.x) * (256 / kGroup)) {
        const int64_t r = item / runs, run = item - r * runs;
        const T* x = static_cast<const T*>(a.x) + r * a.ld;
        T* dx = static_cast<T*>(a.dx) + r * a.ld_dx;
        const uint8_t* mask = kMask ? a.mask + r * a.ld_mask : nullptr;
        const PiecedRow<T> row(x, mask, a.n);
        const int32_t p0 = static_cast<int32_t>(run * kGroup * kPieces);
        uint4 u[kPieces];
        uint32_t bits[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int32_t p = p0 + i * kGroup + t;
            if (p < row.pieces) {
                u[i] = row.load(p);
                if constexpr (kMask) bits[i] = row.active(p);
            }
        }
        const int given = a.T + (a.g_top ? a.k : 0);
        const float m = a.stats[2 * r];
        float sum = 0.f, g;
        for (int i = t; i < given; i += kGroup) {
            given_column(a, r, i, x, mask, m, &g);
            sum += g;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if constexpr (kGroup == 256) {
            if ((t & 31) == 0) sum_of[t >> 5] = sum;
            __syncthreads();
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += sum_of[i];
        }
        const float gh = a.g_entropy ? a.g_entropy[r] : 0.f;
        const GradRow gr{m, a.stats[2 * r + 1], -a.scale * __fmaf_rn(gh, gh != 0.f ? a.entropy[r] : 0.f, sum), -a.scale * gh * kLn2};
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int32_t p = p0 + i * kGroup + t;
            if (p >= row.pieces) continue;
            Piece<T> e;
            e.set(u[i]);
            alignas(16) T o[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float d = gr.dx(e.v[j], a.c);
                o[j] = from_f32<T>(kMask && !(bits[i] >> j & 1) ? 0.f : d);
            }
            const int64_t at = row.column(p);
            if (row.whole(p) && (reinterpret_cast<uintptr_t>(dx + at) & 15) == 0) {
                *reinterpret_cast<uint4*>(dx + at) = *reinterpret_cast<const uint4*>(o);
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (at + j >= 0 && at + j < a.n) dx[at + j] = o[j];
            }
        }
        // the given columns of this run, each by the thread of its first mention
        if constexpr (kGroup == 256) __syncthreads();
        else __syncwarp();
        const int64_t c0 = row.column(p0), c1 = row.column(p0 + kGroup * kPieces);
        for (int i = t; i < given; i += kGroup) {
            const int64_t j = given_column(a, r, i, x, mask, m, &g);
            if (j < 0 || j < c0 || j >= c1) continue;
            bool first = true;
            float own = g;
            for (int e = 0; e < given; ++e) {
                if (e == i) continue;
                float ge;
                if (given_column(a, r, e, x, mask, m, &ge) != j) continue;
                if (e < i) { first = false; break; }
                own += ge;
            }
            if (first) dx[j] = from_f32<T>(__fmaf_rn(a.scale, own, gr.dx(to_f32(x[j]), a.c)));
        }
        if constexpr (kGroup == 256) __syncthreads();
    }
}

}  // namespace maxsim
