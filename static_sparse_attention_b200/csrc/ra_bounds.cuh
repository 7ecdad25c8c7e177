// ra_bounds.cuh -- the debug build's bounds checks (-DRA_DEBUG_BOUNDS) for the kernels
// around the attention, which have no bounded waits and so no abort flag: a global
// offset is held against its buffer's size before use; a failed check records
// RA_ERR_DEVICE_BOUNDS with its site in the error word and the caller skips the access.
// The release build compiles the checks away.
#pragma once
#include <cuda_runtime.h>

#include "ra_internal.h"

namespace ra {

enum : int {
    SITE_I_ROPE = 80, SITE_I_IN, SITE_I_OUT, SITE_I_GRAD_IN, SITE_I_GRAD_OUT, SITE_I_PART, SITE_I_CODE, SITE_I_SCALE,
    SITE_I_QUERY, SITE_I_RESULT
};

// Whether elements [at, at + n) lie in a buffer of `size`.
__device__ __forceinline__ bool inside(int* err, long long at, long long n, long long size, int site)
{
#ifdef RA_DEBUG_BOUNDS
    if (at >= 0 && at + n <= size)
        return true;
    if (atomicCAS(err, 0, static_cast<int>(RA_ERR_DEVICE_BOUNDS)) == 0) {
        err[1] = site;
        err[2] = static_cast<int>(blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z));
    }
    return false;
#else
    (void)err, (void)at, (void)n, (void)size, (void)site;
    return true;
#endif
}

// The error word that a launch of the debug build records in (none in the release build:
// these calls last microseconds).
inline ra_status bounds_word(int** err)
{
#ifdef RA_DEBUG_BOUNDS
    return device_error_word(err);
#else
    *err = nullptr;
    return RA_OK;
#endif
}

}  // namespace ra
