// ar_heads_common.h -- pieces the kernels on attention heads share.
#pragma once

#include "ar_heads.h"
#include "ar_norm_common.h"

namespace ar {

__device__ inline uint32_t divide(uint32_t n, const FastDiv& d)
{
    return (uint32_t)((uint64_t)n * d.mul >> d.shift);
}

// ---- angles -----------------------------------------------------------------

// Cosine and sine of p f.  The angle is taken in 64 bits, in quarter turns,
// and the nearest whole number of those taken off: what is left is exact there
// and becomes a float32 angle of at most pi / 4, where the Taylor series up to
// the 10th power is off by less than 2e-9.  (float32 angles lose a position of
// 100,000 to 2^-8 radians.)
__device__ inline float2 cos_sin(double position, double frequency)
{
    const double q = position * (frequency * 0.63661977236758134308);  // 2 / pi
    const double n = rint(q);
    const float x = (float)((q - n) * 1.57079632679489661923);
    const float x2 = x * x;
    float s = fmaf(x2, 2.75573192e-6f, -1.98412698e-4f);
    s = fmaf(x2, s, 8.33333333e-3f);
    s = fmaf(x2, s, -1.66666667e-1f);
    s = fmaf(x2 * x, s, x);
    float c = fmaf(x2, -2.75573192e-7f, 2.48015873e-5f);
    c = fmaf(x2, c, -1.38888889e-3f);
    c = fmaf(x2, c, 4.16666667e-2f);
    c = fmaf(x2, c, -0.5f);
    c = fmaf(x2, c, 1.0f);
    const int quarter = (int)(n - 4.0 * floor(n * 0.25));
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    return make_float2(quarter == 1 || quarter == 2 ? -a : a, quarter >= 2 ? -b : b);
}

// Cosines and sines, times the factor, of tokens [first, first + count), counted
// over all batches and below `end` (further ones get the last one's):
// [count][slots].  All threads of a workgroup; a barrier has to follow.
__device__ inline void fill_angles(const Turn& t, const FastDiv& tokens, uint32_t first,
                                   uint32_t count, uint32_t end, float2* table)
{
    for (uint32_t i = threadIdx.x; i < count * t.slots; i += blockDim.x) {
        const uint32_t k = divide(i, t.per_slot), pair = i - k * t.slots;
        uint32_t token = first + k;
        token = token < end ? token : end - 1;
        const uint32_t b = divide(token, tokens);
        const uint64_t at = b * t.position_stride + (token - b * tokens.by);
        const double p = t.wide ? (double)static_cast<const int64_t*>(t.positions)[at]
                                : (double)static_cast<const int32_t*>(t.positions)[at];
        const float2 cs = cos_sin(p, t.frequencies[pair < t.pairs ? pair : t.pairs - 1]);
        table[i] = make_float2(cs.x * t.factor, cs.y * (t.factor * t.sign));
    }
}

// ---- a head's elements in registers -------------------------------------------

// W consecutive elements of T in one access, at any element's alignment.
template <class T, int W>
struct Chunk;
template <int W>
struct Chunk<float, W> {
    typedef uint32_t type __attribute__((ext_vector_type(W), aligned(4)));
};
template <>
struct Chunk<float, 1> {
    typedef uint32_t type;
};
template <>
struct Chunk<uint16_t, 8> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Chunk<uint16_t, 4> {
    typedef uint32_t type __attribute__((ext_vector_type(2), aligned(2)));
};
template <>
struct Chunk<uint16_t, 2> {
    typedef uint32_t type __attribute__((aligned(2)));
};
template <>
struct Chunk<uint16_t, 1> {
    typedef uint16_t type;
};

// A unit is two vectors of W elements that a thread rotates together: j and
// the one half a rotation behind it in the layout of halves, else neighbours.
// Unit j's pairs are [j W, (j + 1) W) in both layouts; a thread has units lane,
// lane + lanes, ...
template <class E, int W>
struct Head {
    using T = typename E::T;
    using Raw = typename Chunk<T, W>::type;
    static constexpr int UNITS = kHeadPerLane / (2 * W);

    // Vectors of unit j.
    static __device__ uint2 vectors(uint32_t j, uint32_t turned, int layout)
    {
        return layout == AR_ROTARY_HALVES && j < turned ? make_uint2(j, j + turned)
                                                        : make_uint2(2 * j, 2 * j + 1);
    }

    static __device__ void widen(const Raw& r, float* o)
    {
        if constexpr (sizeof(T) == 4) {
            if constexpr (W == 1) {
                o[0] = __uint_as_float(r);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    o[i] = __uint_as_float(r[i]);
            }
        } else if constexpr (W == 1) {
            o[0] = E::widen(r);
        } else if constexpr (W == 2) {
            o[0] = __uint_as_float(r << 16);
            o[1] = __uint_as_float(r & 0xffff0000u);
        } else {
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                o[2 * i] = __uint_as_float(r[i] << 16);
                o[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
            }
        }
    }

    static __device__ uint32_t two(float a, float b)
    {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const f32x2 f = {a, b};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
    }

    static __device__ Raw narrow(const float* v)
    {
        Raw r;
        if constexpr (sizeof(T) == 4) {
            if constexpr (W == 1) {
                r = __float_as_uint(v[0]);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    r[i] = __float_as_uint(v[i]);
            }
        } else if constexpr (W == 1) {
            r = (uint16_t)two(v[0], v[0]);
        } else if constexpr (W == 2) {
            r = two(v[0], v[1]);
        } else {
#pragma unroll
            for (int i = 0; i < W / 2; ++i)
                r[i] = two(v[2 * i], v[2 * i + 1]);
        }
        return r;
    }

    Raw raw[UNITS][2];

    // Vectors past a head's end are read where its last one is (and not used).
    __device__ void load(const T* p, uint32_t lane, uint32_t lanes, uint32_t nvec, uint32_t turned,
                         int layout)
    {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const uint2 v = vectors(k * lanes + lane, turned, layout);
            const uint32_t a = v.x < nvec ? v.x : nvec - 1, b = v.y < nvec ? v.y : nvec - 1;
            raw[k][0] = __builtin_nontemporal_load(reinterpret_cast<const Raw*>(p + a * W));
            raw[k][1] = __builtin_nontemporal_load(reinterpret_cast<const Raw*>(p + b * W));
        }
    }

    // Their values; 0 past the end.
    __device__ void get(float (&o)[kHeadPerLane], uint32_t lane, uint32_t lanes, uint32_t nvec,
                        uint32_t turned, int layout) const
    {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const uint2 v = vectors(k * lanes + lane, turned, layout);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float* to = o + (2 * k + h) * W;
                widen(raw[k][h], to);
                if ((h ? v.y : v.x) >= nvec)
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        to[i] = 0.0f;
            }
        }
    }

    // Writes values, rounded.
    template <bool NT>
    static __device__ void put(T* p, const float (&o)[kHeadPerLane], uint32_t lane, uint32_t lanes,
                               uint32_t nvec, uint32_t turned, int layout)
    {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const uint2 v = vectors(k * lanes + lane, turned, layout);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = h ? v.y : v.x;
                if (at < nvec) {
                    const Raw r = narrow(o + (2 * k + h) * W);
                    if constexpr (NT)
                        __builtin_nontemporal_store(r, reinterpret_cast<Raw*>(p + at * W));
                    else
                        *reinterpret_cast<Raw*>(p + at * W) = r;
                }
            }
        }
    }

    // Rotates values by a token's table.  A unit of neighbours may be rotated in
    // part: a pair past the last one stays as it is.
    static __device__ void turn(float (&o)[kHeadPerLane], const float2* table, uint32_t lane,
                                uint32_t lanes, uint32_t turned, uint32_t pairs, int layout)
    {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const uint32_t j = k * lanes + lane;
            if (j < turned) {
                float2 cs[W];
#pragma unroll
                for (int i = 0; i < W; ++i)
                    cs[i] = table[j * W + i];
                float* u = o + 2 * k * W;
                if (layout == AR_ROTARY_HALVES) {
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const float a = u[i], b = u[W + i];
                        u[i] = fmaf(cs[i].x, a, -(cs[i].y * b));
                        u[W + i] = fmaf(cs[i].x, b, cs[i].y * a);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const float a = u[2 * i], b = u[2 * i + 1];
                        if (j * W + i < pairs) {
                            u[2 * i] = fmaf(cs[i].x, a, -(cs[i].y * b));
                            u[2 * i + 1] = fmaf(cs[i].x, b, cs[i].y * a);
                        }
                    }
                }
            }
        }
    }

    // Calls f(k, element): where value k of a thread lies in its head.
    template <class F>
    static __device__ void each(uint32_t lane, uint32_t lanes, uint32_t nvec, uint32_t turned,
                                int layout, F f)
    {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const uint2 v = vectors(k * lanes + lane, turned, layout);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = h ? v.y : v.x;
                if (at < nvec)
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        f((2 * k + h) * W + i, at * W + i);
            }
        }
    }
};

__device__ inline float lanes_total(float v, uint32_t lanes)
{
    return lanes < 64 ? lanes_sum(v, lanes) : wave_sum(v);
}

// r of a head's values over `lanes` threads.
__device__ inline float head_rstd(const float (&o)[kHeadPerLane], uint32_t lanes, uint32_t dim,
                                  float eps)
{
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kHeadPerLane; ++i)
        ss = fmaf(o[i], o[i], ss);
    return inv_rms(lanes_total(ss, lanes), dim, eps, [&] {
        double d = 0.0;
#pragma unroll
        for (int i = 0; i < kHeadPerLane; ++i)
            d += (double)o[i] * (double)o[i];
        return lanes_sum(d, lanes);
    });
}

}  // namespace ar
