// Host-side checks that the C entry points share.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "../../include/mxfp4.h"

namespace mx {

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline bool in_range(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

inline mxfp4_status_t check_device()
{
    // gfx950 check, cached per device ordinal: 0 = unknown, 1 = gfx950, 2 = other
    static std::atomic<int> cache[64];
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return MXFP4_ERR_DEVICE;
    if (dev < 64) {
        const int known = cache[dev].load(std::memory_order_relaxed);
        if (known) return known == 1 ? MXFP4_OK : MXFP4_ERR_DEVICE;
    }
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MXFP4_ERR_DEVICE;
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < 64) cache[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
    return ok ? MXFP4_OK : MXFP4_ERR_DEVICE;
}

inline mxfp4_status_t from_hip(hipError_t e) { return e == hipSuccess ? MXFP4_OK : MXFP4_ERR_LAUNCH; }

inline bool valid_in(int t) { return t == MXFP4_IN_F32 || t == MXFP4_IN_BF16; }
inline size_t in_size(int t) { return t == MXFP4_IN_BF16 ? 2 : 4; }
inline bool valid_out(int t) { return t == MXFP4_OUT_F32 || t == MXFP4_OUT_BF16; }
inline size_t out_size(int t) { return t == MXFP4_OUT_BF16 ? 2 : 4; }

// an E4M3 output with rows of length L
inline mxfp4_status_t check_fp8_out(const uint8_t *q, int64_t ldq, const uint8_t *s, int64_t lds, int64_t L)
{
    if (ldq < (L + 127) / 128 * 128 || lds < (L + 127) / 128 || lds < 1) return MXFP4_ERR_ARG;
    if (!s) return MXFP4_ERR_NULL;
    if (!aligned(q, 16) || ldq % 16 != 0) return MXFP4_ERR_ALIGN;
    return MXFP4_OK;
}

}  // namespace mx
