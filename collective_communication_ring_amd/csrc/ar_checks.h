// ar_checks.h -- argument checks that the operators' host sides share.
#pragma once

#include <hip/hip_runtime.h>

#include "ar_internal.h"

namespace ar {

constexpr size_t kMaxElems = (size_t)1 << 46;  // sizes above are refused: no byte offset wraps

inline size_t size_of(int dtype) { return dtype == AR_E4M3 ? 1 : dtype == AR_BF16 ? 2 : 4; }

inline bool stream_type(int dtype) { return dtype == AR_FLOAT32 || dtype == AR_BF16; }

inline bool misaligned(const void* p, int dtype) { return (uintptr_t)p % size_of(dtype) != 0; }

// The status of an operator's launches.
inline int done(hipError_t e)
{
    if (e == hipSuccess)
        return AR_SUCCESS;
    g_util_hip_error = (int)e;
    return AR_ERR_HIP;
}

}  // namespace ar
