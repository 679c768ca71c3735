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

template <class E, bool Q>
void launch_any(const NormArgs& a, hipStream_t s)
{
    const uint64_t grid = std::min<uint64_t>(a.rows, 1u << 16);
    hipLaunchKernelGGL((k_norm_any<E, Q>), dim3((unsigned)grid), dim3(kBlock), 0, s, a);
}

}  // namespace

hipError_t launch_rmsnorm(int dtype, bool e4m3, const NormArgs& a, hipStream_t s)
{
    if (dtype == AR_BF16)
        e4m3 ? launch_any<Elem<AR_BF16>, true>(a, s) : launch_any<Elem<AR_BF16>, false>(a, s);
    else
        e4m3 ? launch_any<Elem<AR_FLOAT32>, true>(a, s) : launch_any<Elem<AR_FLOAT32>, false>(a, s);
    return hipGetLastError();
}

}  // namespace ar
