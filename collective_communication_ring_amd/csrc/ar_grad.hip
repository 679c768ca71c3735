// ar_grad.hip -- the global 2-norm of many tensors, and their scaling by it.
//
// A launch takes a table of spans in its kernel arguments.  The tiles of all
// its spans are numbered through; a workgroup takes a contiguous range of
// them, so it looks its first span up once and then walks on.
//
// Squares are added in float64: every square of a float32 or bfloat16 is exact
// there (48 bits or fewer) and inside its range, so the sum needs no scaling.
#include "ar_norm_common.h"

namespace ar {
namespace {

constexpr uint32_t kIsBf16 = 0x80000000u;

// The span that holds tile `t`: the last whose first tile is <= t.
template <class Table>
__device__ inline int span_of(const Table& tab, uint32_t t)
{
    int lo = 0, hi = tab.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((tab.first[mid] & ~kIsBf16) <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

template <class E>
__device__ inline double sum_tile(const void* src, uint64_t n, uint32_t tile)
{
    using T = typename E::T;
    constexpr uint64_t V = E::VEC;
    const T* p = static_cast<const T*>(src);
    const uint64_t lo = (uint64_t)tile * kGradTileVecs * V;
    const uint64_t hi = lo + kGradTileVecs * V < n ? lo + kGradTileVecs * V : n;
    double acc = 0.0;
    for (uint64_t i = lo + threadIdx.x; i < hi; i += kBlock) {
        const double v = (double)E::widen(p[i]);
        acc = fma(v, v, acc);
    }
    return acc;
}

__global__ __launch_bounds__(kBlock) void k_grad_norm(SpanTable tab, double* partial, int live,
                                                      uint32_t* ticket, float* norm)
{
    constexpr int W = kBlock / 64;
    __shared__ double s_d[W];
    __shared__ uint32_t s_last;
    const uint32_t lo = (uint32_t)((uint64_t)tab.tiles * blockIdx.x / gridDim.x);
    const uint32_t hi = (uint32_t)((uint64_t)tab.tiles * (blockIdx.x + 1) / gridDim.x);
    double acc = 0.0;
    if (lo < hi) {
        int s = span_of(tab, lo);
        for (uint32_t t = lo; t < hi; ++t) {
            while (s + 1 < tab.n && (tab.first[s + 1] & ~kIsBf16) <= t)
                ++s;
            const uint32_t first = tab.first[s];
            const uint32_t tile = t - (first & ~kIsBf16);
            acc += first & kIsBf16 ? sum_tile<Elem<AR_BF16>>(tab.src[s], tab.count[s], tile)
                                   : sum_tile<Elem<AR_FLOAT32>>(tab.src[s], tab.count[s], tile);
        }
    }
    acc = block_sum<W>(acc, s_d);
    // the slot is published before the ticket is taken (release), and whoever
    // takes the last ticket sees every slot (acquire)
    if (threadIdx.x == 0) {
        if ((int)blockIdx.x < live)
            acc += partial[blockIdx.x];
        __hip_atomic_store(partial + blockIdx.x, acc, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = 0;
        if (norm)
            s_last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                     gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last)
        return;
    const int slots = live > (int)gridDim.x ? live : (int)gridDim.x;
    double sum = 0.0;
    for (int i = threadIdx.x; i < slots; i += kBlock)
        sum += __hip_atomic_load(partial + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sum = block_sum<W>(sum, s_d);
    if (threadIdx.x == 0) {
        *norm = (float)sqrt(sum);
        __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

template <class E>
__device__ inline void clip_tile(const void* src, void* dst, uint64_t n, uint32_t tile, float coef)
{
    using T = typename E::T;
    constexpr uint64_t V = E::VEC;
    const T* p = static_cast<const T*>(src);
    T* q = static_cast<T*>(dst);
    const uint64_t lo = (uint64_t)tile * kGradTileVecs * V;
    const uint64_t hi = lo + kGradTileVecs * V < n ? lo + kGradTileVecs * V : n;
    for (uint64_t i = lo + threadIdx.x; i < hi; i += kBlock)
        q[i] = E::narrow(E::widen(p[i]) * coef);
}

__global__ __launch_bounds__(kBlock) void k_grad_clip(SpanPairTable tab, const float* norm,
                                                      float max_norm)
{
    const uint32_t lo = (uint32_t)((uint64_t)tab.tiles * blockIdx.x / gridDim.x);
    const uint32_t hi = (uint32_t)((uint64_t)tab.tiles * (blockIdx.x + 1) / gridDim.x);
    if (lo >= hi)
        return;
    const float nv = *norm;
    const float c = max_norm / (nv + 1e-6f);
    const float coef = nv != nv ? nv : c < 1.0f ? c : 1.0f;
    int s = span_of(tab, lo);
    for (uint32_t t = lo; t < hi; ++t) {
        while (s + 1 < tab.n && (tab.first[s + 1] & ~kIsBf16) <= t)
            ++s;
        if (coef == 1.0f && tab.src[s] == tab.dst[s])
            continue;  // in place, unchanged
        const uint32_t first = tab.first[s];
        const uint32_t tile = t - (first & ~kIsBf16);
        if (first & kIsBf16)
            clip_tile<Elem<AR_BF16>>(tab.src[s], tab.dst[s], tab.count[s], tile, coef);
        else
            clip_tile<Elem<AR_FLOAT32>>(tab.src[s], tab.dst[s], tab.count[s], tile, coef);
    }
}

}  // namespace

hipError_t launch_grad_norm(const SpanTable& t, double* partial, int live, int grid,
                            uint32_t* ticket, float* norm, hipStream_t s)
{
    hipLaunchKernelGGL(k_grad_norm, dim3(grid), dim3(kBlock), 0, s, t, partial, live, ticket, norm);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const SpanPairTable& t, const float* norm, float max_norm, int grid,
                            hipStream_t s)
{
    hipLaunchKernelGGL(k_grad_clip, dim3(grid), dim3(kBlock), 0, s, t, norm, max_norm);
    return hipGetLastError();
}

}  // namespace ar
