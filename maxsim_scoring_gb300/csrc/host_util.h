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

}  // namespace maxsim
