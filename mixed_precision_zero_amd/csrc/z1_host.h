// z1_host.h -- checks that the host code of the operators (z1_ops_api.hip,
// z1_layers_api.hip) shares.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "z1_ops.h"

namespace z1 {
namespace host {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int current_device()
{
    int d = -1;
    if (hipGetDevice(&d) != hipSuccess) {
        (void)hipGetLastError();
        return -1;
    }
    return d;
}

// True when `stream` is a stream of GPU `dev` and that GPU is current.
inline bool runs_on(int dev, z1_stream stream)
{
    if (dev < 0 || current_device() != dev)
        return false;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (!s || s == hipStreamLegacy || s == hipStreamPerThread)
        return true;
    hipDevice_t d = -1;
    if (hipStreamGetDevice(s, &d) != hipSuccess) {
        (void)hipGetLastError();
        return false;
    }
    return d == dev;
}

inline bool is_finite(double x) { return isfinite(x); }

inline size_t type_size(int32_t dtype) { return dtype == Z1_F32 ? 4 : 2; }
inline bool dtype_ok(int32_t t) { return t == Z1_F32 || t == Z1_BF16 || t == Z1_F16; }
inline bool itype_ok(int32_t t) { return t == Z1_I64 || t == Z1_I32; }
inline size_t itype_size(int32_t t) { return t == Z1_I64 ? 8 : 4; }

}  // namespace host
}  // namespace z1
