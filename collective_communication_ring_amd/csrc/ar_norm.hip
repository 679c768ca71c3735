// ar_norm.hip -- RMS norm of the residual stream, alone or behind the
// reduction of the ranks' partial sums.
//
//   h = sum of parts + residual;  r = 1 / sqrt(mean(h^2) + eps);  v = h r w
//
// float32 throughout; sum, y and the scales are each rounded once.
#include <algorithm>

#include "ar_norm_common.h"

namespace ar {
namespace {

// Vectors of a call up to which its rows are spread over as many waves as they
// can use (one vector a thread): 16 waves on each CU.  Below, that is faster
// (bf16 513 x 2048: 4.5 us, two vectors a thread 5.2; 8 ranks' 8 x 4096: 4.1
// and 5.0), above, two vectors are (8192 x 8192: 75 us, one 95; 8193 x 2571: 33
// us, one 37).  Four are for the longest rows alone (8193 x 2571: 38 us).
constexpr uint64_t kFewVecs = 256 * 16 * 64;

// Any row length, one workgroup per row, an element at a time: pass 1 sums the
// squares, pass 2 writes; e4m3 takes the groups' largest values between them.
// Each pass reads the row again (from L2, except the first).  A thread reads
// an element before it writes that element's outputs, and no other thread
// touches it, so an output may be an input's array.
//
// For rows of less than a vector, and the longest: two- and four-byte accesses
// keep it from memory's rate (float32 4096 x 18,432 with residual: 412 us for
// 1.2 GB, 2.9 TB/s; bf16 2048 x 40,000: 676 us for 0.66 GB).
template <class E, bool Q>
__global__ __launch_bounds__(kBlock) void k_norm_any(NormArgs a)
{
    using T = typename E::T;
    constexpr int W = kBlock / 64;
    __shared__ float s_f[W];
    __shared__ double s_d[W];
    __shared__ uint32_t s_u[W];
    const T* x = static_cast<const T*>(a.x);
    const T* res = static_cast<const T*>(a.residual);
    for (uint64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
        const int owner = a.parts > 1 ? (int)(t / a.tokens_per_rank) : 0;
        auto value = [&](uint32_t c) -> float {
            float h;
            if (a.parts > 1) {
                int p = owner;
                for (int i = 0; i < a.parts; ++i) {
                    p = p + 1 == a.parts ? 0 : p + 1;
                    const float v = E::widen(x[(uint64_t)p * a.part_stride + t * a.x_stride + c]);
                    h = i ? h + v : v;
                }
                h /= a.divisor;
            } else {
                h = E::widen(x[t * a.x_stride + c]);
            }
            return res ? h + E::widen(res[t * a.res_stride + c]) : h;
        };
        float ss = 0.0f;
        for (uint32_t c = threadIdx.x; c < a.cols; c += kBlock) {
            const float h = value(c);
            ss = fmaf(h, h, ss);
        }
        ss = block_sum<W>(ss, s_f);
        const float r = inv_rms(ss, a.cols, a.eps, [&] {
            double d = 0.0;
            for (uint32_t c = threadIdx.x; c < a.cols; c += kBlock) {
                const double h = (double)value(c);
                d = fma(h, h, d);
            }
            return block_sum<W>(d, s_d);
        });
        if (a.rstd && threadIdx.x == 0)
            a.rstd[t] = r;
        auto normed = [&](uint32_t c, float h) {
            return h * r * weight_at<E>(a.weight, a.weight_f32, c);
        };
        T* sum = static_cast<T*>(a.sum);
        if constexpr (Q) {
            uint8_t* y = static_cast<uint8_t*>(a.y);
            // whole row: every thread a part of it; else a wave per group
            const bool whole = a.groups == 1;
            const uint32_t lane = whole ? threadIdx.x : threadIdx.x & 63u;
            const uint32_t step = whole ? (uint32_t)kBlock : 64u;
            for (uint32_t g = whole ? 0u : threadIdx.x >> 6; g < a.groups; g += whole ? 1u : W) {
                const uint32_t lo = g * a.group;
                const uint32_t hi = a.cols - lo < a.group ? a.cols : lo + a.group;
                uint32_t m = 0;
                for (uint32_t c = lo + lane; c < hi; c += step) {
                    const uint32_t u = __float_as_uint(normed(c, value(c))) & 0x7fffffffu;
                    m = u > m ? u : m;
                }
                m = whole ? block_umax<W>(m, s_u) : wave_umax(m);
                const float scale = e4m3_scale(m);
                if (lane == 0)
                    a.scale[t * a.groups + g] = scale;
                for (uint32_t c = lo + lane; c < hi; c += step) {
                    const float h = value(c);
                    y[t * a.y_stride + c] = e4m3(normed(c, h) / scale);
                    if (sum)
                        sum[t * a.sum_stride + c] = E::narrow(h);
                }
            }
        } else {
            T* y = static_cast<T*>(a.y);
            for (uint32_t c = threadIdx.x; c < a.cols; c += kBlock) {
                const float h = value(c);
                y[t * a.y_stride + c] = E::narrow(normed(c, h));
                if (sum)
                    sum[t * a.sum_stride + c] = E::narrow(h);
            }
        }
    }
}

// A row's vectors from registers.  The exact and the other case, and the two
// kinds of store, are told apart once for all of them: tested at each store
// they cost bf16 8192 x 8192 81 us instead of 75.
template <class E, int NV>
__device__ inline void store_row(typename E::T* p, const float (&v)[NV][E::VEC], uint32_t lane,
                                 const NormArgs& a)
{
    if (a.exact && a.stream) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            store_whole<E, true>(p + (k * a.lanes + lane) * E::VEC, narrow_slot<E>(v[k]));
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            store_vec<E, false>(p, narrow_slot<E>(v[k]), (k * a.lanes + lane) * E::VEC, a.cols);
    }
}

// Rows of at least a vector that fit in registers: a.lanes threads per row (a
// power of two below 64, or 64 for each of its waves), NV vectors per thread,
// vector k of thread l at column (k lanes + l) VEC.  A workgroup is one row of
// several waves, or as many shorter rows as 256 threads hold.  One pass: every
// input is read once, all loads of a row in flight together, and h stays in
// registers through the sum of squares and the groups' largest values.  A
// thread has read its own elements of all inputs before it writes them, and no
// other thread uses them, so an output may be an input's array.
//
// Bound by memory: bf16 8192 x 8192 with residual and e4m3 output moves its 472
// MB in 75 us (6.3 TB/s; a copy of 1 GiB: 5.9), 8 ranks' 2048 x 8192 reduced and
// normed to e4m3 their 353 MB in 61 us (5.8 TB/s).
template <class E, bool WF32, bool Q, int NV, bool MULTI>
__global__ __launch_bounds__(64 * kMaxWaves) void k_norm(NormArgs a)
{
    using T = typename E::T;
    constexpr int V = E::VEC;
    __shared__ float s_f[kMaxWaves];
    __shared__ double s_d[kMaxWaves];
    __shared__ uint32_t s_u[kMaxWaves];
    const uint32_t lanes = a.lanes, wave = threadIdx.x >> 6;
    const uint32_t lane = lanes <= 64 ? threadIdx.x & (lanes - 1) : threadIdx.x;
    const uint64_t t = a.row0 + (lanes <= 64 ? (blockIdx.x * blockDim.x + threadIdx.x) / lanes
                                             : blockIdx.x);
    if (t >= a.rows)  // all threads of a row; rows of several waves have no such workgroup
        return;
    const auto column = [&](int k) { return (k * lanes + lane) * V; };
    const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
    float h[NV][V];
    u32x4 res[NV];
    Weight<E, WF32> w[NV];
    if (a.residual) {
        const T* r = static_cast<const T*>(a.residual) + t * a.res_stride;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            res[k] = load_vec<E>(r, column(k), a.cols);
    }
    if constexpr (MULTI) {
        // U ranks' vectors in flight at a time (as many as the registers of 1024
        // threads hold), added in the ring's order
        constexpr int U = NV >= 4 ? 1 : NV >= 2 ? 4 : 8;
        int p = (int)(t / a.tokens_per_rank);
        for (int i0 = 0; i0 < a.parts; i0 += U) {
            u32x4 raw[U][NV];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u < a.parts) {
                    p = p + 1 == a.parts ? 0 : p + 1;
                    const T* q = x + (uint64_t)p * a.part_stride;
#pragma unroll
                    for (int k = 0; k < NV; ++k)
                        raw[u][k] = load_vec<E>(q, column(k), a.cols);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u < a.parts) {
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        float v[V];
                        if (!a.exact)
                            fit<E>(raw[u][k], column(k), a.cols);
                        widen_slot<E, V>(raw[u][k], v);
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            h[k][i] = i0 + u ? h[k][i] + v[i] : v[i];
                    }
                }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
            w[k].load(a.weight, column(k), a.cols);
        if (a.divisor != 1.0f)
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    h[k][i] /= a.divisor;
    } else {
        u32x4 raw[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k)
            raw[k] = load_vec<E>(x, column(k), a.cols);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            w[k].load(a.weight, column(k), a.cols);
        if (!a.exact)
#pragma unroll
            for (int k = 0; k < NV; ++k)
                fit<E>(raw[k], column(k), a.cols);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            widen_slot<E, V>(raw[k], h[k]);
    }
    if (!a.exact)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            w[k].fit_to(column(k), a.cols);
            if (a.residual)
                fit<E>(res[k], column(k), a.cols);
        }
    if (a.residual)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float v[V];
            widen_slot<E, V>(res[k], v);
#pragma unroll
            for (int i = 0; i < V; ++i)
                h[k][i] += v[i];
        }
    if (a.sum)
        store_row<E, NV>(static_cast<T*>(a.sum) + t * a.sum_stride, h, lane, a);
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i)
            ss = fmaf(h[k][i], h[k][i], ss);
    ss = row_total(ss, s_f, wave, lanes);
    const float r = inv_rms(ss, a.cols, a.eps, [&] {
        double d = 0.0;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i)
                d = fma((double)h[k][i], (double)h[k][i], d);
        return row_total(d, s_d, wave, lanes);
    });
    if (a.rstd && lane == 0)
        a.rstd[t] = r;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        float v[V];
        w[k].get(v);
#pragma unroll
        for (int i = 0; i < V; ++i)
            h[k][i] = h[k][i] * r * v[i];
    }
    if constexpr (Q) {
        uint8_t* y = static_cast<uint8_t*>(a.y) + t * a.y_stride;
        uint32_t m[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            m[k] = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                // past the row's end: 0, or NaN where r is infinite or NaN
                if (column(k) + i < a.cols)
                    m[k] = umax(m[k], __float_as_uint(h[k][i]) & 0x7fffffffu);
        }
        if (a.groups == 1) {
            uint32_t all = m[0];
#pragma unroll
            for (int k = 1; k < NV; ++k)
                all = umax(all, m[k]);
            all = row_umax(all, s_u, wave, lanes);
#pragma unroll
            for (int k = 0; k < NV; ++k)
                m[k] = all;
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                m[k] = lanes_umax(m[k], a.group / V);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t c = column(k);
            const float scale = e4m3_scale(m[k]);
            if (c < a.cols && c % a.group == 0)
                a.scale[t * a.groups + c / a.group] = scale;
            float quot[V];
            over_scale<V>(h[k], scale, quot);
            u32x4 q = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < V / 4; ++j)
                q[j] = e4m3x4(quot[4 * j], quot[4 * j + 1], quot[4 * j + 2], quot[4 * j + 3]);
            if (c + V <= a.cols) {
                // plain stores also where the others stream: 8 bytes a lane fill
                // half a wave's lines (both streamed: 79 us instead of 75)
                typedef uint32_t u32x2 __attribute__((ext_vector_type(2), aligned(1)));
                typedef uint32_t u32 __attribute__((aligned(1)));
                if constexpr (V == 8)
                    *reinterpret_cast<u32x2*>(y + c) = u32x2{q[0], q[1]};
                else
                    *reinterpret_cast<u32*>(y + c) = q[0];
            } else if (c < a.cols) {
                store_head(y + c, q, a.cols - c);
            }
        }
    } else {
        store_row<E, NV>(static_cast<T*>(a.y) + t * a.y_stride, h, lane, a);
    }
}

template <class E, bool WF32, bool Q, int NV, bool MULTI>
void launch_row(NormArgs a, uint32_t nvec, hipStream_t s)
{
    a.lanes = 64 * ((nvec + 64 * NV - 1) / (64 * NV));
    if (NV == 1)
        while (a.lanes <= 64 && a.lanes / 2 >= nvec && a.lanes > 1)
            a.lanes /= 2;
    a.exact = a.cols == NV * a.lanes * E::VEC;
    const uint32_t rows = a.lanes <= 64 ? kBlock / a.lanes : 1;
    const uint64_t most = kNormMaxThreads / a.lanes;  // a multiple of a workgroup's rows
    for (a.row0 = 0; a.row0 < a.rows; a.row0 += most) {
        const uint64_t n = std::min<uint64_t>(a.rows - a.row0, most);
        hipLaunchKernelGGL((k_norm<E, WF32, Q, NV, MULTI>), dim3((unsigned)((n + rows - 1) / rows)),
                           dim3(a.lanes * rows), 0, s, a);
    }
}

template <class E, bool WF32, bool Q, bool MULTI>
void launch_typed(const NormArgs& a, hipStream_t s)
{
    const uint32_t nvec = (a.cols + E::VEC - 1) / E::VEC;
    // rows of less than a vector and of more than 4096 go an element at a time
    if (a.cols < E::VEC || nvec > 64 * 4 * kMaxWaves)
        hipLaunchKernelGGL((k_norm_any<E, Q>), dim3((unsigned)std::min<uint64_t>(a.rows, 1u << 16)),
                           dim3(kBlock), 0, s, a);
    else if (nvec > 64 * 2 * kMaxWaves)
        launch_row<E, WF32, Q, 4, MULTI>(a, nvec, s);
    else if (nvec <= 64 || (nvec <= 64 * kMaxWaves && a.rows * nvec <= kFewVecs))
        launch_row<E, WF32, Q, 1, MULTI>(a, nvec, s);
    else
        launch_row<E, WF32, Q, 2, MULTI>(a, nvec, s);
}

template <class E, bool WF32, bool Q>
void launch_parts(const NormArgs& a, hipStream_t s)
{
    a.parts > 1 ? launch_typed<E, WF32, Q, true>(a, s) : launch_typed<E, WF32, Q, false>(a, s);
}

template <class E, bool WF32>
void launch_out(bool e4m3, const NormArgs& a, hipStream_t s)
{
    e4m3 ? launch_parts<E, WF32, true>(a, s) : launch_parts<E, WF32, false>(a, s);
}

}  // namespace

hipError_t launch_rmsnorm(int dtype, bool e4m3, NormArgs a, hipStream_t s)
{
    a.stream = a.rows * a.cols * (dtype == AR_BF16 ? 2 : 4) > kStreamBytes;
    if (dtype == AR_FLOAT32)
        launch_out<Elem<AR_FLOAT32>, false>(e4m3, a, s);
    else if (a.weight_f32)
        launch_out<Elem<AR_BF16>, true>(e4m3, a, s);
    else
        launch_out<Elem<AR_BF16>, false>(e4m3, a, s);
    return hipGetLastError();
}

}  // namespace ar
