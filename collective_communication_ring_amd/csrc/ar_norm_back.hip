// ar_norm_back.hip -- backward pass of the RMS norm.
//
//   n = x r,  g = dy w:   dx = r (g - n mean(g n)) + dsum,   dw = sum_t dy n
//
// float32 throughout.  dw's rows are shared out to `blocks` workgroups per
// rank, each leaving one partial row, and a second launch adds those: the
// order depends on sizes alone.
#include <algorithm>

#include "ar_norm_common.h"

namespace ar {
namespace {

// dx, any row length: one workgroup per row, two passes over it.  A thread
// reads an element's dy, x and dsum before it writes its dx.
template <class E>
__global__ __launch_bounds__(kBlock) void k_back_dx_any(NormBackArgs a)
{
    using T = typename E::T;
    constexpr int W = kBlock / 64;
    __shared__ float s_f[W];
    const uint64_t rows = a.rows_per_rank * (uint64_t)a.ranks;
    for (uint64_t t = blockIdx.x; t < rows; t += gridDim.x) {
        const T* dy = static_cast<const T*>(a.dy) + t * a.dy_stride;
        const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
        const T* ds = a.dsum ? static_cast<const T*>(a.dsum) + t * a.dsum_stride : nullptr;
        T* dx = static_cast<T*>(a.dx) + t * a.dx_stride;
        const float r = a.rstd[t];
        float dot = 0.0f;
        for (uint32_t c = threadIdx.x; c < a.cols; c += kBlock) {
            const float g = E::widen(dy[c]) * weight_at<E>(a.weight, a.weight_f32, c);
            dot = fmaf(g, E::widen(x[c]) * r, dot);
        }
        const float m = block_sum<W>(dot, s_f) / (float)a.cols;
        for (uint32_t c = threadIdx.x; c < a.cols; c += kBlock) {
            const float g = E::widen(dy[c]) * weight_at<E>(a.weight, a.weight_f32, c);
            float d = r * (g - E::widen(x[c]) * r * m);
            if (ds)
                d += E::widen(ds[c]);
            dx[c] = E::narrow(d);
        }
    }
}

// dw's partial rows: a thread per column, a block of rows per workgroup.
template <class E>
__global__ __launch_bounds__(kBlock) void k_back_dw_any(NormBackArgs a)
{
    using T = typename E::T;
    const uint32_t c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.cols)
        return;
    const int b = blockIdx.y, rank = blockIdx.z;
    const uint64_t base = (uint64_t)rank * a.rows_per_rank;
    const uint64_t lo = base + a.rows_per_rank * b / a.blocks;
    const uint64_t hi = base + a.rows_per_rank * (b + 1) / a.blocks;
    float acc = 0.0f;
    for (uint64_t t = lo; t < hi; ++t)
        acc = fmaf(E::widen(static_cast<const T*>(a.dy)[t * a.dy_stride + c]),
                   E::widen(static_cast<const T*>(a.x)[t * a.x_stride + c]) * a.rstd[t], acc);
    a.partial[((uint64_t)rank * a.blocks + b) * a.cols + c] = acc;
}

// dweight[rank] = the sum of its partial rows (none: zeros).
__global__ __launch_bounds__(kBlock) void k_back_dw_join(const float* partial, float* dweight,
                                                         uint32_t cols, int blocks)
{
    const uint32_t c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= cols)
        return;
    const float* p = partial + (uint64_t)blockIdx.y * blocks * cols + c;
    float acc = 0.0f;
    for (int b = 0; b < blocks; ++b)
        acc += p[(uint64_t)b * cols];
    dweight[(uint64_t)blockIdx.y * cols + c] = acc;
}

template <class E>
void launch_any(const NormBackArgs& a, hipStream_t s)
{
    const uint64_t rows = a.rows_per_rank * (uint64_t)a.ranks;
    const unsigned col_blocks = (a.cols + kBlock - 1) / kBlock;
    // dw first: it reads dy and x, which dx may overwrite
    hipLaunchKernelGGL(k_back_dw_any<E>, dim3(col_blocks, a.blocks, a.ranks), dim3(kBlock), 0, s, a);
    hipLaunchKernelGGL(k_back_dx_any<E>, dim3((unsigned)std::min<uint64_t>(rows, 1u << 16)),
                       dim3(kBlock), 0, s, a);
}

}  // namespace

int norm_back_blocks(uint64_t rows_per_rank, int ranks)
{
    const uint64_t want = std::max<uint64_t>(1, (uint64_t)kNormBackMaxBlocks / ranks);
    return (int)std::min<uint64_t>(rows_per_rank, want);
}

hipError_t launch_rmsnorm_back(int dtype, const NormBackArgs& a, hipStream_t s)
{
    if (a.blocks) {
        if (dtype == AR_BF16)
            launch_any<Elem<AR_BF16>>(a, s);
        else
            launch_any<Elem<AR_FLOAT32>>(a, s);
    }
    hipLaunchKernelGGL(k_back_dw_join, dim3((a.cols + kBlock - 1) / kBlock, a.ranks), dim3(kBlock), 0,
                       s, a.partial, a.dweight, a.cols, a.blocks);
    return hipGetLastError();
}

}  // namespace ar
