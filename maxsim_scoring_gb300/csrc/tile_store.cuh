// What the matrix products' tile kernels share: bounded waits, the epilogue's
// tensor-memory loads and packed arithmetic, and the way of a warp's 16-bit
// outputs from registers to memory.
#pragma once

#include <cstdint>

#include "head_kernels.cuh"
#include "ptx.cuh"

namespace maxsim {

constexpr int kTileStatusTimeout = 4;  // MAXSIM_ERR_TIMEOUT

// Bounded wait of a thread: gives up after the limit (recorded in the device
// status word) or when another role of the CTA has.
template <bool kCluster = false, typename Args, typename Ctl>
__device__ __forceinline__ bool tile_wait(const Args& a, Ctl* ctl, uint64_t* bar_ptr, uint32_t parity) {
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

template <bool kCluster = false, typename Args, typename Ctl>
__device__ __forceinline__ bool tile_wait_warp(const Args& a, Ctl* ctl, uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, tile_wait<kCluster>(a, ctl, bar, parity));
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

// Stores a warp's 32 rows of A x kCols columns along B of 16-bit outputs, which
// its lanes hold (a row each). `out` is the matrix, ld its stride; row_n rows
// exist from ra0 on, rows_b columns in all, rb0 is the first one. `stage` is the
// warp's staging (4 KB, no longer in use).
template <typename T, int kCols, bool kSwap, bool kTma>
__device__ __forceinline__ void store_held(const uint32_t (&held)[kCols / 32][16], uint8_t* stage, T* out, int64_t ld, int64_t ra0,
                                           int64_t rb0, int64_t rows_b, int row_n, const CUtensorMap* tm_out) {
    constexpr int kChunks = kCols / 32;
    const int lane = threadIdx.x & 31;
    if (row_n <= 0) return;
    const bool in_a = lane < row_n;
    __syncwarp();  // the table is done with
    if constexpr (kSwap) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int64_t rb = rb0 + c * 32;
            const int n = static_cast<int>(min(static_cast<int64_t>(32), rows_b - rb));
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
            if (n0 >= rows_b) break;
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
            if (lane == 0) tma_store_2d(tm_out, smem_u32(stage), static_cast<int32_t>(n0), static_cast<int32_t>(ra0));
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
            if (n0 >= rows_b) break;
            const int left = static_cast<int>(min(static_cast<int64_t>(kRun), rows_b - n0));
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

}  // namespace maxsim
