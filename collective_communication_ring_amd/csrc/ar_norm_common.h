// ar_norm_common.h -- pieces the norm's forward and backward kernels share.
#pragma once

#include <type_traits>

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

// Sum over aligned runs of `lanes` (a power of two, 32 at most).
__device__ inline float lanes_sum(float v, uint32_t lanes)
{
    if (lanes > 1)
        v += __uint_as_float(dpp<kXor1>(__float_as_uint(v)));
    if (lanes > 2)
        v += __uint_as_float(dpp<kXor2>(__float_as_uint(v)));
    if (lanes > 4)
        v += __uint_as_float(dpp<kMirror8>(__float_as_uint(v)));
    if (lanes > 8)
        v += __uint_as_float(dpp<kMirror16>(__float_as_uint(v)));
    if (lanes > 16)
        v += __shfl_xor(v, 16);
    return v;
}

__device__ inline double lanes_sum(double v, uint32_t lanes)
{
    for (uint32_t d = 1; d < lanes; d <<= 1)
        v += __shfl_xor(v, (int)d);
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

template <int CTRL>
__device__ inline double dpp(double v)
{
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double((long long)((uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32 |
                                            dpp<CTRL>((uint32_t)u)));
}

__device__ inline double lane_of(double v, int lane)
{
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

__device__ inline double wave_sum(double v)
{
    v += dpp<kXor1>(v);
    v += dpp<kXor2>(v);
    v += dpp<kMirror8>(v);
    v += dpp<kMirror16>(v);
    return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
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

// The same over a row's `lanes`: a power of two below 64, or 64 for each of its
// waves (16 at most; the calling one's number is w).  Each array `s` is used
// once between barriers: every lane reads one wave's value, and a fold over 16
// lanes leaves the whole on all.
__device__ inline float row_total(float v, float* s, uint32_t w, uint32_t lanes)
{
    if (lanes < 64)
        return lanes_sum(v, lanes);
    v = wave_sum(v);
    if (lanes == 64)
        return v;
    if ((threadIdx.x & 63u) == 0)
        s[w] = v;
    __syncthreads();
    const uint32_t l = threadIdx.x & 15u;
    return row_sum(l * 64 < lanes ? s[l] : 0.0f);
}

__device__ inline double row_total(double v, double* s, uint32_t w, uint32_t lanes)
{
    if (lanes <= 64)
        return lanes_sum(v, lanes);
    v = wave_sum(v);
    if ((threadIdx.x & 63u) == 0)
        s[w] = v;
    __syncthreads();
    v = 0.0;
    for (uint32_t k = 0; k * 64 < lanes; ++k)
        v += s[k];
    return v;
}

__device__ inline uint32_t row_umax(uint32_t v, uint32_t* s, uint32_t w, uint32_t lanes)
{
    v = lanes_umax(v, lanes < 64 ? lanes : 64u);
    if (lanes <= 64)
        return v;
    if ((threadIdx.x & 63u) == 0)
        s[w] = v;
    __syncthreads();
    const uint32_t l = threadIdx.x & 15u;
    return lanes_umax(l * 64 < lanes ? s[l] : 0u, 16);
}

// r = 1 / sqrt(mean + eps).  A float32 sum of squares that is infinite may
// have overflowed from finite elements, and one this small may have lost all
// of them, where eps does not outweigh that: `again` then takes it in 64 bits.
template <class Again>
__device__ inline float inv_rms(float ss, uint32_t cols, float eps, Again again)
{
    // the same on every thread of the row
    if (ss == __builtin_inff() || (ss < 1e-25f && eps < 1e-20f))
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

// q = v / scale for a group's values, as the float32 division rounds wherever
// that shows in e4m3.  The product with the rounded reciprocal, q0, may be off
// by an ulp, enough to fall on the other side of a border of e4m3; the remainder
// v - q0 scale, exact in one fma, puts it right.  A border has 5 significant
// bits: for every float32 significand of a scale, and the values around every
// border, the result is the division's.  Remainders of small scales would
// underflow: both sides of those are raised by 2^64 first.  An infinite scale
// has no remainder: the quotients are what 0, its reciprocal, makes of the
// values.  (bf16 8192 x 8192 in groups of 128: 75.4 us, 75.1 with q0 alone, 81
// with a division a value; 32 x 8192: 4.92, 4.70, 5.22.)
template <int V>
__device__ inline void over_scale(const float (&v)[V], float scale, float (&q)[V])
{
    const float inv = 1.0f / scale;
    const bool tiny = scale < 0x1p-80f;
    const float up = tiny ? 0x1p64f : 1.0f, down = tiny ? inv * 0x1p-64f : inv;
    const float s = inv == 0.0f ? 0.0f : scale * up;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float q0 = v[i] * inv;
        q[i] = copysignf(fmaf(fmaf(-q0, s, v[i] * up), down, q0), v[i]);  // -0 stays
    }
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

// The vector of elements [c, c + VEC) of a row of `cols` >= VEC elements.  One
// that would reach past the row's end is read where it ends there, so that a
// row's loads are all alike and in flight together; fit() then puts it right,
// where it is used.  (A cut-short vector read element by element cost a row of
// 2571 bfloat16 a third of its time: a chain of waits in its last wave.)
template <class E>
__device__ inline u32x4 load_vec(const typename E::T* p, uint32_t c, uint32_t cols)
{
    const uint32_t at = c + E::VEC <= cols ? c : cols - E::VEC;
    return __builtin_nontemporal_load(
        reinterpret_cast<const typename AnyVec<typename E::T>::type*>(p + at));
}

// Moves what load_vec read for column c there; elements past the end are zero.
template <class E>
__device__ inline void fit(u32x4& r, uint32_t c, uint32_t cols)
{
    if (c + E::VEC <= cols)
        return;
    uint32_t drop = (c < cols ? c + E::VEC - cols : E::VEC) * (uint32_t)sizeof(typename E::T) * 8;
    uint64_t lo = (uint64_t)r[1] << 32 | r[0], hi = (uint64_t)r[3] << 32 | r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (drop >= 64) {
            lo = hi;
            hi = 0;
            drop -= 64;
        }
    if (drop) {
        lo = lo >> drop | hi << (64 - drop);
        hi >>= drop;
    }
    r = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// The first n (< 16 / sizeof(U)) units of a vector, in at most log2 stores.
template <class U>
__device__ inline void store_head(U* p, const u32x4& r, uint32_t n)
{
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2), aligned(1)));
    typedef uint32_t u32 __attribute__((aligned(1)));
    uint64_t left = (uint64_t)r[1] << 32 | r[0];
    if (n * sizeof(U) & 8) {
        *reinterpret_cast<u32x2*>(p) = u32x2{r[0], r[1]};
        p += 8 / sizeof(U);
        left = (uint64_t)r[3] << 32 | r[2];
    }
    uint32_t word = (uint32_t)left;
    if (n * sizeof(U) & 4) {
        *reinterpret_cast<u32*>(p) = word;
        p += 4 / sizeof(U);
        word = (uint32_t)(left >> 32);
    }
    if constexpr (sizeof(U) == 2) {
        if (n & 1)
            *p = (uint16_t)word;
    } else if constexpr (sizeof(U) == 1) {
        typedef uint16_t u16 __attribute__((aligned(1)));
        if (n & 2) {
            *reinterpret_cast<u16*>(p) = (uint16_t)word;
            p += 2;
            word >>= 16;
        }
        if (n & 1)
            *p = (uint8_t)word;
    }
}

// A whole vector stored; NT: not kept in the caches' order of use.
template <class E, bool NT>
__device__ inline void store_whole(typename E::T* p, const u32x4& r)
{
    using Vec = typename AnyVec<typename E::T>::type;
    if constexpr (NT)
        __builtin_nontemporal_store(r, reinterpret_cast<Vec*>(p));
    else
        *reinterpret_cast<Vec*>(p) = r;
}

// Elements [c, c + VEC) of a row of `cols`, as far as it goes.
template <class E, bool NT>
__device__ inline void store_vec(typename E::T* p, const u32x4& r, uint32_t c, uint32_t cols)
{
    if (c + E::VEC <= cols)
        store_whole<E, NT>(p + c, r);
    else if (c < cols)
        store_head(p + c, r, cols - c);
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

// VEC weights from column c of `cols` >= VEC, of the stream's type or float32;
// past the end they are zero.
template <class E, bool WF32>
struct Weight {
    static constexpr int N = WF32 ? E::VEC / 4 : 1;
    using W = typename std::conditional<WF32, Elem<AR_FLOAT32>, E>::type;
    u32x4 r[N];
    __device__ void load(const void* w, uint32_t c, uint32_t cols)
    {
#pragma unroll
        for (int h = 0; h < N; ++h)
            r[h] = load_vec<W>(static_cast<const typename W::T*>(w), c + 4 * h, cols);
    }
    __device__ void fit_to(uint32_t c, uint32_t cols)
    {
#pragma unroll
        for (int h = 0; h < N; ++h)
            fit<W>(r[h], c + 4 * h, cols);
    }
    __device__ void get(float (&o)[E::VEC]) const
    {
#pragma unroll
        for (int h = 0; h < N; ++h) {
            float part[W::VEC];
            widen_slot<W, W::VEC>(r[h], part);
#pragma unroll
            for (int i = 0; i < W::VEC; ++i)
                o[4 * h + i] = part[i];
        }
    }
};

// The weight of column c, float32 or of the stream's type.
template <class E>
__device__ inline float weight_at(const void* w, int f32, uint64_t c)
{
    return f32 ? static_cast<const float*>(w)[c] : E::widen(static_cast<const typename E::T*>(w)[c]);
}

}  // namespace ar
