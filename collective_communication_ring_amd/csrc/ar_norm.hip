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

// Any row length, one workgroup per row, an element at a time: pass 1 sums the
// squares, pass 2 writes; e4m3 takes the groups' largest values between them.
// Each pass reads the row again (from L2, except the first).  A thread reads
// an element before it writes that element's outputs, and no other thread
// touches it, so an output may be an input's array.
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
                const float inv = 1.0f / scale;
                if (lane == 0)
                    a.scale[t * a.groups + g] = scale;
                for (uint32_t c = lo + lane; c < hi; c += step) {
                    const float h = value(c);
                    y[t * a.y_stride + c] = e4m3(normed(c, h) * inv);
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

// Rows that fit in registers: TPR threads per row (64: a wave each, four rows
// to a workgroup), NV vectors per thread, vector k of a row's thread l at
// column (k TPR + l) VEC.  One pass: every input is read once, all loads of a
// row in flight together, and h stays in registers through the sum of squares
// and the groups' largest values.  A thread has read its own elements of all
// inputs before it writes them, and no other thread touches them, so an output
// may be an input's array.
template <class E, bool WF32, bool Q, int TPR, int NV, bool MULTI>
__global__ __launch_bounds__(TPR < kBlock ? kBlock : TPR) void k_norm(NormArgs a)
{
    using T = typename E::T;
    constexpr int V = E::VEC;
    constexpr int W = TPR / 64;
    constexpr int ROWS = TPR < kBlock ? kBlock / TPR : 1;
    __shared__ float s_f[W];
    __shared__ double s_d[W];
    __shared__ uint32_t s_u[W];
    const uint32_t lane = threadIdx.x % TPR;
    const uint64_t t = (uint64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    if (t >= a.rows)  // a whole wave's rows (TPR == 64), never a part of a workgroup's row
        return;
    const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
    float h[NV][V];
    u32x4 res[NV];
    if (a.residual) {
        const T* r = static_cast<const T*>(a.residual) + t * a.res_stride;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            res[k] = load_part<E>(r, (k * TPR + lane) * V, a.cols);
    }
    if constexpr (MULTI) {
        // U ranks' vectors in flight at a time, added in the ring's order
        constexpr int U = NV >= 4 ? (TPR > 512 ? 1 : 2) : NV >= 2 ? 4 : 8;
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
                        raw[u][k] = load_part<E>(q, (k * TPR + lane) * V, a.cols);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u < a.parts) {
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        float v[V];
                        widen_slot<E, V>(raw[u][k], v);
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            h[k][i] = i0 + u ? h[k][i] + v[i] : v[i];
                    }
                }
        }
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
            raw[k] = load_part<E>(x, (k * TPR + lane) * V, a.cols);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            widen_slot<E, V>(raw[k], h[k]);
    }
    float w[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
        load_weight<E, WF32>(a.weight, (k * TPR + lane) * V, a.cols, w[k]);
    if (a.residual)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float v[V];
            widen_slot<E, V>(res[k], v);
#pragma unroll
            for (int i = 0; i < V; ++i)
                h[k][i] += v[i];
        }
    if (a.sum) {
        T* sum = static_cast<T*>(a.sum) + t * a.sum_stride;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            store_part<E>(sum, narrow_slot<E>(h[k]), (k * TPR + lane) * V, a.cols);
    }
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i)
            ss = fmaf(h[k][i], h[k][i], ss);
    ss = block_sum<W>(ss, s_f);
    const float r = inv_rms(ss, a.cols, a.eps, [&] {
        double d = 0.0;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i)
                d = fma((double)h[k][i], (double)h[k][i], d);
        return block_sum<W>(d, s_d);
    });
    if (a.rstd && lane == 0)
        a.rstd[t] = r;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i)
            h[k][i] = h[k][i] * r * w[k][i];
    if constexpr (Q) {
        uint8_t* y = static_cast<uint8_t*>(a.y) + t * a.y_stride;
        uint32_t m[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            m[k] = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                // past the row's end: 0, or NaN where r is infinite or NaN
                if ((k * TPR + lane) * V + i < a.cols)
                    m[k] = umax(m[k], __float_as_uint(h[k][i]) & 0x7fffffffu);
        }
        if (a.groups == 1) {
            uint32_t all = m[0];
#pragma unroll
            for (int k = 1; k < NV; ++k)
                all = umax(all, m[k]);
            all = block_umax<W>(all, s_u);
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
            const uint32_t c = (k * TPR + lane) * V;
            const float scale = e4m3_scale(m[k]);
            const float inv = 1.0f / scale;
            if (c < a.cols && c % a.group == 0)
                a.scale[t * a.groups + c / a.group] = scale;
            uint32_t q[V / 4];
#pragma unroll
            for (int j = 0; j < V / 4; ++j)
                q[j] = e4m3x4(h[k][4 * j] * inv, h[k][4 * j + 1] * inv, h[k][4 * j + 2] * inv,
                              h[k][4 * j + 3] * inv);
            if (c + V <= a.cols) {
                if constexpr (V == 8) {
                    typedef uint32_t u32x2 __attribute__((ext_vector_type(2), aligned(1)));
                    *reinterpret_cast<u32x2*>(y + c) = u32x2{q[0], q[1]};
                } else {
                    typedef uint32_t u32x1 __attribute__((aligned(1)));
                    *reinterpret_cast<u32x1*>(y + c) = q[0];
                }
            } else if (c < a.cols) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (c + i < a.cols)
                        y[c + i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
            }
        }
    } else {
        T* y = static_cast<T*>(a.y) + t * a.y_stride;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            store_part<E>(y, narrow_slot<E>(h[k]), (k * TPR + lane) * V, a.cols);
    }
}

template <class E, bool WF32, bool Q, int TPR, int NV, bool MULTI>
void launch_row(const NormArgs& a, hipStream_t s)
{
    constexpr int threads = TPR < kBlock ? kBlock : TPR;
    constexpr int rows = threads / TPR;
    hipLaunchKernelGGL((k_norm<E, WF32, Q, TPR, NV, MULTI>),
                       dim3((unsigned)((a.rows + rows - 1) / rows)), dim3(threads), 0, s, a);
}

template <class E, bool WF32, bool Q, bool MULTI>
void launch_typed(const NormArgs& a, hipStream_t s)
{
    const uint32_t nvec = (a.cols + E::VEC - 1) / E::VEC;
    // rows past 2^31 workgroups and rows longer than 4096 vectors go an
    // element at a time
    if (a.rows > 1u << 30 || nvec > 4096)
        hipLaunchKernelGGL((k_norm_any<E, Q>), dim3((unsigned)std::min<uint64_t>(a.rows, 1u << 16)),
                           dim3(kBlock), 0, s, a);
    else if (nvec <= 64)
        launch_row<E, WF32, Q, 64, 1, MULTI>(a, s);
    else if (nvec <= 128)
        launch_row<E, WF32, Q, 64, 2, MULTI>(a, s);
    else if (nvec <= 256)
        launch_row<E, WF32, Q, 256, 1, MULTI>(a, s);
    else if (nvec <= 512)
        launch_row<E, WF32, Q, 256, 2, MULTI>(a, s);
    else if (nvec <= 1024)
        launch_row<E, WF32, Q, 256, 4, MULTI>(a, s);
    else if (nvec <= 2048)
        launch_row<E, WF32, Q, 512, 4, MULTI>(a, s);
    else
        launch_row<E, WF32, Q, 1024, 4, MULTI>(a, s);
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

hipError_t launch_rmsnorm(int dtype, bool e4m3, const NormArgs& a, hipStream_t s)
{
    if (dtype == AR_FLOAT32)
        launch_out<Elem<AR_FLOAT32>, false>(e4m3, a, s);
    else if (a.weight_f32)
        launch_out<Elem<AR_BF16>, true>(e4m3, a, s);
    else
        launch_out<Elem<AR_BF16>, false>(e4m3, a, s);
    return hipGetLastError();
}

}  // namespace ar
