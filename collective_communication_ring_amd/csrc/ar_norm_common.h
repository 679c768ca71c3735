// ar_norm_common.h -- pieces the norm's forward and backward kernels share.
#pragma once

#include "ar_elem.h"
#include "ar_internal.h"
#include "ar_ops.h"

namespace ar {

// ---- sums and maxima over lanes ------------------------------------------------

// The value of another lane of the same 16: lane ^ 1, lane ^ 2, the mirror
// image within 8, the mirror image within 16.  Folding over the four in turn
// leaves every lane with its 16's result.  One vector instruction each, where
// a shuffle goes through the LDS crossbar.
template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;

__device__ inline float row_sum(float v)
{
    v += __uint_as_float(dpp<kXor1>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kXor2>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kMirror8>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kMirror16>(__float_as_uint(v)));
    return v;
}

__device__ inline float lane_of(float v, int lane)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}

__device__ inline float wave_sum(float v)
{
    v = row_sum(v);
    return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

__device__ inline double wave_sum(double v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Largest of values compared as unsigned bit patterns, over aligned runs of
// `lanes` (a power of two).  For the bits of |v| that order is the order of
// the values, with NaN above infinity: a NaN or an infinity among the values
// is the result.
__device__ inline uint32_t lanes_umax(uint32_t v, uint32_t lanes)
{
    if (lanes > 1)
        v = umax(v, dpp<kXor1>(v));
    if (lanes > 2)
        v = umax(v, dpp<kXor2>(v));
    if (lanes > 4)
        v = umax(v, dpp<kMirror8>(v));
    if (lanes > 8)
        v = umax(v, dpp<kMirror16>(v));
    if (lanes > 16)
        v = umax(v, (uint32_t)__shfl_xor((int)v, 16));
    if (lanes > 32)
        v = umax(v, (uint32_t)__shfl_xor((int)v, 32));
    return v;
}

__device__ inline uint32_t wave_umax(uint32_t v) { return lanes_umax(v, 64); }

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

// ---- 16-byte vectors at any element alignment ------------------------------------

// gfx950 reads and writes 16 bytes at any element's address in one
// instruction, so a row needs no alignment; the type says so to the compiler.
template <class T>
struct AnyVec {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4)));
};
template <>
struct AnyVec<uint16_t> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};

// Elements [c, c + VEC) of a row of `cols`; those past its end read as zero.
// Only a row's last vector can be cut short, and it goes element by element.
template <class E>
__device__ inline u32x4 load_part(const typename E::T* p, uint32_t c, uint32_t cols)
{
    using T = typename E::T;
    u32x4 r = {0u, 0u, 0u, 0u};
    if (c + E::VEC <= cols) {
        r = __builtin_nontemporal_load(reinterpret_cast<const typename AnyVec<T>::type*>(p + c));
    } else if (c < cols) {
#pragma unroll
        for (int i = 0; i < E::VEC; ++i)
            if (c + i < cols)
                r[i * sizeof(T) / 4] |= E::t_bits(p[c + i]) << (8 * (i * sizeof(T) % 4));
    }
    return r;
}

template <class E>
__device__ inline void store_part(typename E::T* p, const u32x4& r, uint32_t c, uint32_t cols)
{
    using T = typename E::T;
    if (c + E::VEC <= cols) {
        *reinterpret_cast<typename AnyVec<T>::type*>(p + c) = r;
    } else if (c < cols) {
#pragma unroll
        for (int i = 0; i < E::VEC; ++i)
            if (c + i < cols)
                p[c + i] = E::t_from_bits(r[i * sizeof(T) / 4] >> (8 * (i * sizeof(T) % 4)));
    }
}

// VEC float values rounded to a vector of T.
template <class E>
__device__ inline u32x4 narrow_slot(const float (&v)[E::VEC])
{
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (E::VEC == 4) {
            r[i] = __float_as_uint(v[i]);
        } else {
            typedef float f32x2 __attribute__((ext_vector_type(2)));
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            const f32x2 f = {v[2 * i], v[2 * i + 1]};
            r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
        }
    }
    return r;
}

// VEC weights from column c, of the stream's type or float32.
template <class E, bool WF32>
__device__ inline void load_weight(const void* w, uint32_t c, uint32_t cols, float (&o)[E::VEC])
{
    if constexpr (WF32) {
#pragma unroll
        for (int h = 0; h < E::VEC / 4; ++h) {
            float part[4];
            widen_slot<Elem<AR_FLOAT32>, 4>(
                load_part<Elem<AR_FLOAT32>>(static_cast<const float*>(w), c + 4 * h, cols), part);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[4 * h + i] = part[i];
        }
    } else {
        widen_slot<E, E::VEC>(load_part<E>(static_cast<const typename E::T*>(w), c, cols), o);
    }
}

// The weight of column c, float32 or of the stream's type.
template <class E>
__device__ inline float weight_at(const void* w, int f32, uint64_t c)
{
    return f32 ? static_cast<const float*>(w)[c] : E::widen(static_cast<const typename E::T*>(w)[c]);
}

}  // namespace ar
