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

// Cosine and sine of p f, `turns` being f / 2 pi.  The angle is taken in 64 bits,
// in turns, whole turns and then the nearest whole number of quarters taken off:
// what is left is exact there and becomes a float32 angle of at most pi / 4, where
// the Taylor series up to the 10th power is off by less than 2e-9.  (float32 angles
// lose a position of 100,000 to 2^-8 radians.)
__device__ inline float2 cos_sin(double position, double turns)
{
    const double q = 4.0 * __builtin_amdgcn_fract(position * turns);
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
    const int quarter = (int)n;  // 0 .. 4
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    const uint32_t minus_a = (uint32_t)((quarter + 1) & 2) << 30, minus_b = (uint32_t)(quarter & 2) << 30;
    return make_float2(__uint_as_float(__float_as_uint(a) ^ minus_a),
                       __uint_as_float(__float_as_uint(b) ^ minus_b));
}

// Cosines and sines, times the factor, of tokens [first, first + count), counted
// over all batches: [count][pairs].  By and for the lanes of one wave, whose reads
// and writes of LDS keep their order: waves do not wait for each other.  A lane
// takes the same pairs of every token it takes.
__device__ inline void fill_angles(const Turn& t, const FastDiv& tokens, uint32_t first,
                                   uint32_t count, float2* table)
{
    __builtin_amdgcn_wave_barrier();
    const uint32_t sub = (threadIdx.x & 63u) / t.lanes;
    for (uint32_t pair = (threadIdx.x & 63u) - sub * t.lanes; pair < t.pairs; pair += 64) {
        const double turns = t.frequencies[pair] * 0.15915494309189533577;  // 1 / 2 pi
        for (uint32_t k = sub; k < count; k += 64 / t.lanes) {
            const uint32_t b = divide(first + k, tokens);
            const uint64_t at = b * t.position_stride + (first + k - b * tokens.by);
            const double p = t.wide ? (double)static_cast<const int64_t*>(t.positions)[at]
                                    : (double)static_cast<const int32_t*>(t.positions)[at];
            const float2 cs = cos_sin(p, turns);
            table[k * t.pairs + pair] = make_float2(cs.x * t.factor, cs.y * (t.factor * t.sign));
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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

// A thread holds units of two vectors of W elements: of a head's units, numbers
// lane, lane + lanes, ...  In the layout of halves a rotated unit j is vector j and
// the one half a rotation behind it, pairs [j W, (j + 1) W).  Else a pair lies
// within a vector, and a thread's two are `lanes` apart, so that a wave's accesses
// are of whole lines (two neighbours a thread: 16384 x 40 heads of 128 90 us, so
// 59) -- but for single elements, whose neighbour is the pair's other one.
//
// WHOLE: a head's vectors fill its lanes.  Then nothing is conditional: a wait for
// loads that are followed by stores of which there may be any number is a wait for
// these, too, as one counter counts both in order.
template <class E, int W, int LAYOUT, bool WHOLE>
struct Head {
    using T = typename E::T;
    using Raw = typename Chunk<T, W>::type;
    static constexpr int UNITS = kHeadPerLane / (2 * W);
    static constexpr bool HALVES = LAYOUT == AR_ROTARY_HALVES;

    // Vectors of a thread's k-th unit; `turned`: rotated units of a head (halves).
    static __device__ uint2 vectors(int k, uint32_t lane, uint32_t lanes, uint32_t turned)
    {
        const uint32_t j = k * lanes + lane;
        if (HALVES && j < turned)
            return make_uint2(j, j + turned);
        if (HALVES || W == 1)
            return make_uint2(2 * j, 2 * j + 1);
        return make_uint2(j + k * lanes, j + (k + 1) * lanes);
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
    __device__ void load(const T* p, uint32_t lane, uint32_t lanes, uint32_t nvec, uint32_t turned)
    {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const uint2 v = vectors(k, lane, lanes, turned);
            // (the same for every head: taken out of their loop)
            const uint32_t a = WHOLE || v.x < nvec ? v.x : nvec - 1, b = WHOLE || v.y < nvec ? v.y : nvec - 1;
            raw[k][0] = __builtin_nontemporal_load(reinterpret_cast<const Raw*>(p + a * W));
            raw[k][1] = __builtin_nontemporal_load(reinterpret_cast<const Raw*>(p + b * W));
        }
    }

    // All of them one value's bits (of a bfloat16, twice).
    __device__ void set(uint32_t bits)
    {
#pragma unroll
        for (int k = 0; k < UNITS; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if constexpr (W * sizeof(T) <= 4)
                    raw[k][h] = (Raw)bits;
                else
#pragma unroll
                    for (int i = 0; i < (int)(W * sizeof(T)) / 4; ++i)
                        raw[k][h][i] = bits;
    }

    // Their values; 0 past the end.
    __device__ void get(float (&o)[kHeadPerLane], uint32_t lane, uint32_t lanes, uint32_t nvec,
                        uint32_t turned) const
    {
#pragma unroll
        for (int k = 0; k < UNITS; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                widen(raw[k][h], o + (2 * k + h) * W);
        if constexpr (!WHOLE) {
#pragma unroll
            for (int k = 0; k < UNITS; ++k) {
                const uint2 v = vectors(k, lane, lanes, turned);
#pragma unroll
                for (int i = 0; i < 2 * W; ++i)
                    o[2 * k * W + i] = (i < W ? v.x : v.y) < nvec ? o[2 * k * W + i] : 0.0f;
            }
        }
    }

    // Writes values, rounded.  stream: larger than the L2s.
    static __device__ void put(T* p, const float (&o)[kHeadPerLane], uint32_t lane, uint32_t lanes,
                               uint32_t nvec, uint32_t turned, int stream)
    {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const uint2 v = vectors(k, lane, lanes, turned);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = h ? v.y : v.x;
                const Raw r = narrow(o + (2 * k + h) * W);
                if (!WHOLE && at >= nvec)
                    continue;
                if (stream)
                    __builtin_nontemporal_store(r, reinterpret_cast<Raw*>(p + at * W));
                else
                    *reinterpret_cast<Raw*>(p + at * W) = r;
            }
        }
    }

    // Rotates values by a token's table.  A vector of pairs may be rotated in part.
    static __device__ void turn(float (&o)[kHeadPerLane], const float2* table, uint32_t lane,
                                uint32_t lanes, uint32_t turned, uint32_t pairs)
    {
        const auto rotate = [](float& a, float& b, float2 cs) {
            const float x = a;
            a = fmaf(cs.x, x, -(cs.y * b));
            b = fmaf(cs.x, b, cs.y * x);
        };
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            float* u = o + 2 * k * W;
            if constexpr (HALVES) {
                const uint32_t j = k * lanes + lane;
                if (j < turned) {
                    float2 cs[W];
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        cs[i] = table[j * W + i];
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        rotate(u[i], u[W + i], cs[i]);
                }
            } else if constexpr (W == 1) {
                const uint32_t j = k * lanes + lane;
                if (j < pairs)
                    rotate(u[0], u[1], table[j]);
            } else {
                const uint2 v = vectors(k, lane, lanes, turned);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t first = (h ? v.y : v.x) * (W / 2);
                    if (first + W / 2 <= pairs) {
                        float2 cs[W / 2];
#pragma unroll
                        for (int i = 0; i < W / 2; ++i)
                            cs[i] = table[first + i];
#pragma unroll
                        for (int i = 0; i < W / 2; ++i)
                            rotate(u[h * W + 2 * i], u[h * W + 2 * i + 1], cs[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < W / 2; ++i)
                            if (first + i < pairs)
                                rotate(u[h * W + 2 * i], u[h * W + 2 * i + 1], table[first + i]);
                    }
                }
            }
        }
    }

    // Calls f(k, element): where value k of a thread lies in its head.
    template <class F>
    static __device__ void each(uint32_t lane, uint32_t lanes, uint32_t nvec, uint32_t turned, F f)
    {
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const uint2 v = vectors(k, lane, lanes, turned);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = h ? v.y : v.x;
                if (WHOLE || at < nvec)
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        f((2 * k + h) * W + i, at * W + i);
            }
        }
    }
};

// Reads a word of every 64 bytes of a kernel's arguments at once: a line of them
// that is first read where it is needed costs a trip to memory there.
template <class Args>
__device__ inline void touch(const Args& a)
{
    const uint32_t* words = reinterpret_cast<const uint32_t*>(&a);
#pragma unroll
    for (size_t i = 0; i < sizeof(Args) / 4; i += 16)
        __asm__ __volatile__("" ::"s"(words[i]));
}

// Both sides' weights on their way to LDS, [2][dim], by a workgroup of 256: read
// early, written behind other loads' waits.
template <class E>
struct Weights {
    float w[2];
    __device__ void load(const void* const (&from)[2], int f32, uint32_t dim)
    {
#pragma unroll
        for (int side = 0; side < 2; ++side)
            w[side] = from[side] && threadIdx.x < dim ? weight_at<E>(from[side], f32, threadIdx.x) : 0.0f;
    }
    __device__ void store(const void* const (&from)[2], int f32, uint32_t dim, float* to) const
    {
        for (int side = 0; side < 2; ++side) {
            if (threadIdx.x < dim)
                to[side * dim + threadIdx.x] = w[side];
            for (uint32_t c = threadIdx.x + 256; from[side] && c < dim; c += 256)
                to[side * dim + c] = weight_at<E>(from[side], f32, c);
        }
    }
};

// Calls f(c) with c the widest vector of elements of E that `width` allows for,
// and whether a head's `nvec` of them fill its lanes.
template <int V, bool B>
struct Width {
    static constexpr int value = V;
    static constexpr bool whole = B;
};
template <class E, class F>
void with_width(int width, bool whole, F f)
{
    if (width == E::VEC && whole)
        f(Width<E::VEC, true>{});
    else if (width == E::VEC)
        f(Width<E::VEC, false>{});
    else if (E::VEC > 4 && width == 4)
        f(Width<4, false>{});
    else if (width == 2)
        f(Width<2, false>{});
    else
        f(Width<1, false>{});
}

__device__ inline float lanes_total(float v, uint32_t lanes)
{
    return lanes < 64 ? lanes_sum(v, lanes) : wave_sum(v);
}

// r of a head's values over `lanes` threads: by the hardware's reciprocal root,
// off by 2^-23 of it at most.  A float32 sum of squares that is infinite may have
// overflowed from finite elements, and one this small may have lost all of them,
// where eps does not outweigh that: it is taken again in 64 bits.
__device__ inline float head_rstd(const float (&o)[kHeadPerLane], uint32_t lanes, uint32_t dim,
                                  float per_dim, float eps)
{
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kHeadPerLane; ++i)
        ss = fmaf(o[i], o[i], ss);
    ss = lanes_total(ss, lanes);
    // the same on every thread of the head
    if (__builtin_expect(ss == __builtin_inff() || (ss < 1e-25f && eps < 1e-20f), 0)) {
        double d = 0.0;
#pragma unroll
        for (int i = 0; i < kHeadPerLane; ++i)
            d += (double)o[i] * (double)o[i];
        return (float)(1.0 / sqrt(lanes_sum(d, lanes) / (double)dim + (double)eps));
    }
    return __builtin_amdgcn_rsqf(fmaf(ss, per_dim, eps));
}

}  // namespace ar
