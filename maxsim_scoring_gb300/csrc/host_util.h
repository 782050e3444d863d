// What the host sides of the library's translation units share: the device's
// properties, the device status word and the TMA descriptor encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "maxsim.h"

namespace maxsim {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s bound on any single device-side wait
constexpr size_t kSmemBudget = 232448;          // 227 KB: opt-in shared memory per block on sm_100 / sm_103
constexpr int64_t kI32Max = 2147483647;

struct HostDevice {
    int index = 0;
    int num_sms = 0;
    int smem_optin = 0;
    int* status = nullptr;  // device status word
    EncodeTiledFn encode = nullptr;
};

// The current device, checked to be one that the library is built for.
maxsim_status host_device(HostDevice* out);

// Workspace of maxsim_linear_int8, or (size_t)-1 for an invalid shape.
size_t linear_int8_ws_bytes(int64_t M, int64_t N, int64_t K, int64_t ld_x, int64_t ld_w);

inline bool ptr_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t bytes_round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline int elem_bytes(maxsim_dtype t) { return t == MAXSIM_F32 ? 4 : 2; }
inline bool any_dtype(maxsim_dtype t) { return t == MAXSIM_F16 || t == MAXSIM_BF16 || t == MAXSIM_F32; }

// A [rows, cols] operand with rows ld elements apart whose bytes can be addressed with 64 bits.
inline bool rows_fit(int64_t rows, int64_t cols, int64_t ld) {
    return ld >= cols && (rows <= 1 || ld <= (int64_t(1) << 60) / std::max<int64_t>(rows, 1));
}

// Blocks for `items`, per_block each, at most `most` (their kernels stride).
inline unsigned grid_of(int64_t items, int64_t per_block, int64_t most) {
    return static_cast<unsigned>(std::max<int64_t>(1, std::min((items + per_block - 1) / per_block, most)));
}

inline maxsim_status launched() { return cudaGetLastError() == cudaSuccess ? MAXSIM_OK : MAXSIM_ERR_CUDA; }

}  // namespace maxsim
