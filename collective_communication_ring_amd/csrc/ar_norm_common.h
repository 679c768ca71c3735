// ar_norm_common.h -- pieces the norm's forward and backward kernels share.
#pragma once

#include "ar_elem.h"
#include "ar_internal.h"
#include "ar_ops.h"

namespace ar {

__device__ inline float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

__device__ inline double wave_sum(double v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

// Largest of values compared as unsigned bit patterns.  For the bits of |v|
// that order is the order of the values, with NaN above infinity: a NaN or an
// infinity among the values is the result.
__device__ inline uint32_t wave_umax(uint32_t v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint32_t o = __shfl_xor(v, d);
        v = o > v ? o : v;
    }
    return v;
}

// Sum over a workgroup of W waves, the same bits on every thread.  `s` is
// shared memory of W values; the call may follow another on the same `s`.
template <int W, class F>
__device__ inline F block_sum(F v, F* s)
{
    v = wave_sum(v);
    if constexpr (W > 1) {
        __syncthreads();
        if ((threadIdx.x & 63u) == 0)
            s[threadIdx.x >> 6] = v;
        __syncthreads();
        v = s[0];
#pragma unroll
        for (int w = 1; w < W; ++w)
            v += s[w];
    }
    return v;
}

template <int W>
__device__ inline uint32_t block_umax(uint32_t v, uint32_t* s)
{
    v = wave_umax(v);
    if constexpr (W > 1) {
        __syncthreads();
        if ((threadIdx.x & 63u) == 0)
            s[threadIdx.x >> 6] = v;
        __syncthreads();
        v = s[0];
#pragma unroll
        for (int w = 1; w < W; ++w)
            v = s[w] > v ? s[w] : v;
    }
    return v;
}

// r = 1 / sqrt(mean + eps).  A float32 sum of squares that is infinite may
// have overflowed from finite elements: `again` then takes it in 64 bits.
template <class Again>
__device__ inline float inv_rms(float ss, uint32_t cols, float eps, Again again)
{
    if (ss == __builtin_inff())  // the same on every thread of the row
        return (float)(1.0 / sqrt(again() / (double)cols + (double)eps));
    return 1.0f / sqrtf(ss / (float)cols + eps);
}

constexpr float kE4M3Max = 448.0f;
constexpr float kE4M3MinScale = 1.17549435e-38f;  // 2^-126: its reciprocal is finite

// A group's scale from the bits of its largest |v| (NaN stays NaN).
__device__ inline float e4m3_scale(uint32_t amax_bits)
{
    const float s = __uint_as_float(amax_bits) / kE4M3Max;
    return s < kE4M3MinScale ? kE4M3MinScale : s;
}

// Four values to four e4m3 bytes, to nearest even.  |q| is at most 448 plus a
// rounding (it was divided by its group's scale), which rounds to 448; an
// infinity or NaN becomes NaN.
__device__ inline uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint32_t r = 0;
    r = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)r, false);
    r = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, (int)r, true);
    return r;
}

__device__ inline uint8_t e4m3(float a)
{
    return (uint8_t)((uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, a, 0, false) & 0xffu);
}

// The weight of column c, float32 or of the stream's type.
template <class E>
__device__ inline float weight_at(const void* w, int f32, uint64_t c)
{
    return f32 ? static_cast<const float*>(w)[c] : E::widen(static_cast<const typename E::T*>(w)[c]);
}

}  // namespace ar
