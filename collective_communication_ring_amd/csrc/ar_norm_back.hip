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

// Row t of an operand.
template <class E>
__device__ inline const typename E::T* row_of(const void* p, uint64_t t, uint64_t stride)
{
    return static_cast<const typename E::T*>(p) + t * stride;
}

template <class E, bool WF32>
__device__ inline void weight_vec(const NormBackArgs& a, uint32_t c, float (&o)[E::VEC])
{
    Weight<E, WF32> raw;
    raw.load(a.weight, c, a.cols);
    if (!a.exact)
        raw.fit_to(c, a.cols);
    raw.get(o);
}

template <class E>
__device__ inline void get_vec(const NormBackArgs& a, u32x4 r, uint32_t c, float (&o)[E::VEC])
{
    if (!a.exact)
        fit<E>(r, c, a.cols);
    widen_slot<E, E::VEC>(r, o);
}

// dot += g n and acc += dy n over a vector.
template <int V>
__device__ inline void forward_of(const float (&x)[V], const float (&dy)[V], const float (&w)[V],
                                  float r, float* dot, float (&acc)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float n = x[j] * r;
        *dot = fmaf(dy[j] * w[j], n, *dot);
        acc[j] = fmaf(dy[j], n, acc[j]);
    }
}

// r (g - n m) over a vector.
template <int V>
__device__ inline void backward_of(const float (&x)[V], const float (&dy)[V], const float (&w)[V],
                                   float r, float m, float (&d)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j)
        d[j] = r * (dy[j] * w[j] - x[j] * r * m);
}

// A row's vector of dx.
template <class E>
__device__ inline void store_dx(const NormBackArgs& a, uint64_t t, uint32_t c,
                                const float (&d)[E::VEC])
{
    typename E::T* p = static_cast<typename E::T*>(a.dx) + t * a.dx_stride;
    if (a.exact && a.stream)
        store_whole<E, true>(p + c, narrow_slot<E>(d));
    else
        store_vec<E, false>(p, narrow_slot<E>(d), c, a.cols);
}

template <int V>
__device__ inline void load_acc(const float4* s, uint32_t stride, float (&o)[V])
{
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
        const float4 f = s[h * stride];
        o[4 * h] = f.x, o[4 * h + 1] = f.y, o[4 * h + 2] = f.z, o[4 * h + 3] = f.w;
    }
}

template <int V>
__device__ inline void store_acc(float4* s, uint32_t stride, const float (&v)[V])
{
#pragma unroll
    for (int h = 0; h < V / 4; ++h)
        s[h * stride] = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
}

template <int V>
__device__ inline void store_partial(float* p, const float (&v)[V], uint32_t c, uint32_t cols)
{
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
        const float part[4] = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
        store_vec<Elem<AR_FLOAT32>, false>(p, narrow_slot<Elem<AR_FLOAT32>>(part), c + 4 * h, cols);
    }
}

// An operand's vectors in flight.
template <int NV>
struct BackRow {
    u32x4 x[NV], dy[NV], ds[NV];
    float r;
};

template <class E, int NV>
__device__ inline void load_row(const NormBackArgs& a, uint64_t t, uint32_t lane, uint32_t lanes,
                                BackRow<NV>& o)
{
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const uint32_t c = (k * lanes + lane) * E::VEC;
        o.x[k] = load_vec<E>(row_of<E>(a.x, t, a.x_stride), c, a.cols);
        o.dy[k] = load_vec<E>(row_of<E>(a.dy, t, a.dy_stride), c, a.cols);
    }
    if (a.dsum)
#pragma unroll
        for (int k = 0; k < NV; ++k)
            o.ds[k] = load_vec<E>(row_of<E>(a.dsum, t, a.dsum_stride),
                                  (k * lanes + lane) * E::VEC, a.cols);
    o.r = a.rstd[t];
}

// Rows of a vector to 1024 vectors: a vector per thread, `lanes` threads per row
// (a power of two below 64, or 64 for each of its waves) and `rows` rows side
// by side in a workgroup.  One pass: dy, x and dsum are read once, and a
// workgroup keeps the weight and its own sums for dw in registers while it
// takes rows b rows, (b + blocks) rows, ... of its rank, the next one's loads
// in flight while one is reduced (two ahead: no faster).  A row is read whole
// before it is written, by the threads that write it, so dx may be an input's
// array.
//
// Bound by memory: bf16 8192 x 8192 with dsum moves its 537 MB in 91 us with
// the join (5.9 TB/s, as a copy of 1 GiB).
template <class E, bool WF32>
__global__ __launch_bounds__(64 * kMaxWaves) void k_back(NormBackArgs a)
{
    constexpr int V = E::VEC;
    __shared__ float s_f[2][kMaxWaves];
    __shared__ float4 s_dw[64 * (kMaxWaves - 1) * V / 4];
    const uint32_t lanes = a.lanes, wave = threadIdx.x >> 6, waves = lanes >> 6;
    const uint32_t sub = threadIdx.x / lanes;  // which of the workgroup's rows
    const uint32_t lane = threadIdx.x - sub * lanes, c = lane * V;
    const uint64_t base = (uint64_t)blockIdx.y * a.rows_per_rank;
    const uint64_t step = (uint64_t)gridDim.x * a.rows;
    uint64_t i = (uint64_t)blockIdx.x * a.rows + sub;
    BackRow<1> cur, next;
    if (i < a.rows_per_rank)
        load_row<E>(a, base + i, lane, lanes, cur);
    float w[V], acc[V];
    weight_vec<E, WF32>(a, c, w);
#pragma unroll
    for (int j = 0; j < V; ++j)
        acc[j] = 0.0f;
    // every thread makes every turn, also one without a row (i - sub is the
    // workgroup's first row): they meet at the barrier
    for (int turn = 0; i - sub < a.rows_per_rank; i += step, turn ^= 1) {
        const bool on = i < a.rows_per_rank;
        if (i + step < a.rows_per_rank)
            load_row<E>(a, base + i + step, lane, lanes, next);
        float x[V], dy[V], dot = 0.0f;
        if (on) {
            get_vec<E>(a, cur.x[0], c, x);
            get_vec<E>(a, cur.dy[0], c, dy);
            forward_of<V>(x, dy, w, cur.r, &dot, acc);
        }
        if (lanes < 64) {
            dot = lanes_sum(dot, lanes);
        } else {
            dot = wave_sum(dot);
            if (waves > 1) {
                // the two halves of s_f take turns: a wave is at most one row ahead
                if ((threadIdx.x & 63u) == 0)
                    s_f[turn][wave] = dot;
                __syncthreads();
                const uint32_t l = threadIdx.x & 15u;
                dot = row_sum(l < waves ? s_f[turn][sub * waves + l] : 0.0f);
            }
        }
        if (on) {
            float d[V];
            backward_of<V>(x, dy, w, cur.r, dot / (float)a.cols, d);
            if (a.dsum) {
                float ds[V];
                get_vec<E>(a, cur.ds[0], c, ds);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    d[j] += ds[j];
            }
            store_dx<E>(a, base + i, c, d);
        }
        cur = next;
    }
    // the workgroup's rows: one partial row.  First those that share a wave,
    // then what is left over `span` threads each.
    for (uint32_t d = lanes; d < 64; d <<= 1)
#pragma unroll
        for (int j = 0; j < V; ++j)
            acc[j] += __shfl_xor(acc[j], (int)d);
    const uint32_t span = lanes < 64 ? 64 : lanes, group = threadIdx.x / span;
    const uint32_t at = threadIdx.x - group * span, groups = blockDim.x / span;
    if (group)
        store_acc<V>(s_dw + (group - 1) * (V / 4) * span + at, span, acc);
    __syncthreads();
    if (group || at >= lanes)
        return;
    for (uint32_t o = 0; o + 1 < groups; ++o) {
        float v[V];
        load_acc<V>(s_dw + o * (V / 4) * span + at, span, v);
#pragma unroll
        for (int j = 0; j < V; ++j)
            acc[j] += v[j];
    }
    store_partial<V>(a.partial + ((uint64_t)blockIdx.y * gridDim.x + blockIdx.x) * a.cols, acc, c,
                     a.cols);
}

// Longer rows, NV vectors per thread of a workgroup of 1024 (128 registers
// each): the sums for dw lie in LDS, and the weight is read again for every row
// (from L2).  HOLD: the row stays in registers, with the next one's loads in
// flight.  Else it is read twice, the second time out of the caches; all of its
// first reads come before its writes, and the second ones are of what the same
// thread writes.
//
// float32 4096 x 8192 with dsum 116 us (4.6 TB/s), bf16 2048 x 16,384 69 us (3.9
// TB/s), 2048 x 32,768 159 us (3.4 TB/s): besides the rows, the weight's reads
// and the sums' in LDS for every row, and the partial rows.
template <class E, bool WF32, int NV, bool HOLD>
__global__ __launch_bounds__(64 * kMaxWaves) void k_back_long(NormBackArgs a)
{
    using T = typename E::T;
    constexpr int V = E::VEC;
    constexpr uint32_t L = 64 * kMaxWaves;
    __shared__ float s_f[2][kMaxWaves];
    __shared__ float4 s_dw[L * NV * V / 4];
    const uint32_t lane = threadIdx.x, wave = lane >> 6;
    const uint64_t base = (uint64_t)blockIdx.y * a.rows_per_rank;
    for (int q = 0; q < NV * V / 4; ++q)
        s_dw[q * L + lane] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    BackRow<HOLD ? NV : 1> cur, next;
    if (HOLD && blockIdx.x < a.rows_per_rank)
        load_row<E>(a, base + blockIdx.x, lane, L, cur);
    int turn = 0;
    for (uint64_t i = blockIdx.x; i < a.rows_per_rank; i += gridDim.x, turn ^= 1) {
        const uint64_t t = base + i;
        const T* xr = row_of<E>(a.x, t, a.x_stride);
        const T* dyr = row_of<E>(a.dy, t, a.dy_stride);
        if (HOLD && i + gridDim.x < a.rows_per_rank)
            load_row<E>(a, t + gridDim.x, lane, L, next);
        const float r = HOLD ? cur.r : a.rstd[t];
        float dot = 0.0f;
        const auto sums = [&](uint32_t k, const u32x4& rx, const u32x4& rdy) {
            const uint32_t c = (k * L + lane) * V;
            float x[V], dy[V], w[V], acc[V];
            float4* s = s_dw + k * (V / 4) * L + lane;
            weight_vec<E, WF32>(a, c, w);
            load_acc<V>(s, L, acc);
            get_vec<E>(a, rx, c, x);
            get_vec<E>(a, rdy, c, dy);
            forward_of<V>(x, dy, w, r, &dot, acc);
            store_acc<V>(s, L, acc);
        };
        if constexpr (HOLD) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                sums(k, cur.x[k], cur.dy[k]);
        } else {
#pragma unroll 2
            for (uint32_t k = 0; k * L * V < a.cols; ++k) {
                const uint32_t c = (k * L + lane) * V;
                sums(k, load_vec<E>(xr, c, a.cols), load_vec<E>(dyr, c, a.cols));
            }
        }
        dot = wave_sum(dot);
        if ((lane & 63u) == 0)
            s_f[turn][wave] = dot;
        __syncthreads();
        const float m = row_sum(s_f[turn][lane & 15u]) / (float)a.cols;
        const auto write = [&](uint32_t k, const u32x4& rx, const u32x4& rdy, const u32x4& rds) {
            const uint32_t c = (k * L + lane) * V;
            float x[V], dy[V], w[V], d[V];
            weight_vec<E, WF32>(a, c, w);
            get_vec<E>(a, rx, c, x);
            get_vec<E>(a, rdy, c, dy);
            backward_of<V>(x, dy, w, r, m, d);
            if (a.dsum) {
                float ds[V];
                get_vec<E>(a, rds, c, ds);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    d[j] += ds[j];
            }
            store_dx<E>(a, t, c, d);
        };
        if constexpr (HOLD) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                write(k, cur.x[k], cur.dy[k], cur.ds[k]);
            cur = next;
        } else {
#pragma unroll 2
            for (uint32_t k = 0; k * L * V < a.cols; ++k) {
                const uint32_t c = (k * L + lane) * V;
                const u32x4 rx = load_vec<E>(xr, c, a.cols), rdy = load_vec<E>(dyr, c, a.cols);
                u32x4 rds = rx;
                if (a.dsum)
                    rds = load_vec<E>(row_of<E>(a.dsum, t, a.dsum_stride), c, a.cols);
                write(k, rx, rdy, rds);
            }
        }
    }
    float* p = a.partial + ((uint64_t)blockIdx.y * gridDim.x + blockIdx.x) * a.cols;
    for (uint32_t k = 0; k * L * V < a.cols; ++k) {
        float acc[V];
        load_acc<V>(s_dw + k * (V / 4) * L + lane, L, acc);
        store_partial<V>(p, acc, (k * L + lane) * V, a.cols);
    }
}

// dweight[rank] = the sum of its partial rows (none: zeros): 32 columns to a
// workgroup, their rows dealt to 8 groups of threads.
constexpr int kJoinCols = 32;
__global__ __launch_bounds__(kBlock) void k_back_dw_join(const float* partial, float* dweight,
                                                         uint32_t cols, int blocks)
{
    constexpr int G = kBlock / kJoinCols;
    __shared__ float s_f[G][kJoinCols];
    const uint32_t col = threadIdx.x % kJoinCols, g = threadIdx.x / kJoinCols;
    const uint32_t c = blockIdx.x * kJoinCols + col;
    float acc = 0.0f;
    if (c < cols) {
        const float* p = partial + (uint64_t)blockIdx.y * blocks * cols + c;
#pragma unroll 8
        for (int b = g; b < blocks; b += G)
            acc += p[(uint64_t)b * cols];
    }
    s_f[g][col] = acc;
    __syncthreads();
    if (g || c >= cols)
        return;
#pragma unroll
    for (int o = 1; o < G; ++o)
        acc += s_f[o][col];
    dweight[(uint64_t)blockIdx.y * cols + c] = acc;
}

void join(const NormBackArgs& a, int blocks, hipStream_t s)
{
    hipLaunchKernelGGL(k_back_dw_join, dim3((a.cols + kJoinCols - 1) / kJoinCols, a.ranks),
                       dim3(kBlock), 0, s, a.partial, a.dweight, a.cols, blocks);
}

// `launch` with its partial rows' place: dweight itself where there is only one.
template <class Launch>
void with_join(NormBackArgs a, int blocks, hipStream_t s, Launch launch)
{
    float* partial = a.partial;
    if (blocks == 1)
        a.partial = a.dweight;
    launch(a);
    a.partial = partial;
    if (blocks > 1)
        join(a, blocks, s);
}

template <class E, bool WF32>
void launch_row(NormBackArgs a, uint32_t nvec, hipStream_t s)
{
    a.lanes = (nvec + 63) / 64 * 64;
    while (a.lanes <= 64 && a.lanes / 2 >= nvec && a.lanes > 1)
        a.lanes /= 2;
    a.exact = a.cols == a.lanes * E::VEC;
    // as many rows side by side as 16 waves hold, but no more than leave each of
    // `blocks` workgroups its own (whole waves of them).  Where one workgroup
    // takes a rank's rows in two turns, it does, without the join's launch (8
    // ranks' 4 x 1024 bf16: 5.6 -> 4.1 us; two turns: even).
    const uint64_t side = 64 * kMaxWaves / a.lanes;
    const uint64_t share = a.rows_per_rank <= 2 * side ? a.rows_per_rank
                                                       : (a.rows_per_rank + a.blocks - 1) / a.blocks;
    const uint32_t unit = a.lanes < 64 ? 64 / a.lanes : 1;
    a.rows = (uint32_t)std::min<uint64_t>(side, (share + unit - 1) / unit * unit);
    if (a.rows_per_rank <= 2 * side)
        a.blocks = 1;
    const int blocks = (int)std::min<uint64_t>((a.rows_per_rank + a.rows - 1) / a.rows, a.blocks);
    with_join(a, blocks, s, [&](const NormBackArgs& b) {
        hipLaunchKernelGGL((k_back<E, WF32>), dim3(blocks, a.ranks), dim3(a.lanes * a.rows), 0, s, b);
    });
}

template <class E, bool WF32, int NV, bool HOLD>
void launch_long(NormBackArgs a, hipStream_t s)
{
    a.exact = a.cols == 64 * kMaxWaves * NV * E::VEC;
    if (a.rows_per_rank <= 2)
        a.blocks = 1;  // as in launch_row
    with_join(a, a.blocks, s, [&](const NormBackArgs& b) {
        hipLaunchKernelGGL((k_back_long<E, WF32, NV, HOLD>), dim3(a.blocks, a.ranks),
                           dim3(64 * kMaxWaves), 0, s, b);
    });
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
    join(a, a.blocks, s);
}

template <class E, bool WF32>
void launch_typed(const NormBackArgs& a, hipStream_t s)
{
    const uint32_t nvec = (a.cols + E::VEC - 1) / E::VEC;
    if (a.cols < E::VEC || nvec > 64 * 4 * kMaxWaves)
        launch_any<E>(a, s);  // rows of less than a vector, and of more than 4096
    else if (nvec <= 64 * kMaxWaves)
        launch_row<E, WF32>(a, nvec, s);
    else if (nvec <= 64 * 2 * kMaxWaves)
        launch_long<E, WF32, 2, !WF32>(a, s);  // float32 weights beside bfloat16: too many registers
    else
        launch_long<E, WF32, 4, false>(a, s);
}

}  // namespace

int norm_back_blocks(uint64_t rows_per_rank, int ranks)
{
    const uint64_t want = std::max<uint64_t>(1, (uint64_t)kNormBackMaxBlocks / ranks);
    return (int)std::min<uint64_t>(rows_per_rank, want);
}

hipError_t launch_rmsnorm_back(int dtype, NormBackArgs a, hipStream_t s)
{
    a.stream = a.rows_per_rank * a.ranks * a.cols * (dtype == AR_BF16 ? 2 : 4) > kStreamBytes;
    if (!a.rows_per_rank)
        join(a, 0, s);
    else if (dtype == AR_FLOAT32)
        launch_typed<Elem<AR_FLOAT32>, false>(a, s);
    else if (a.weight_f32)
        launch_typed<Elem<AR_BF16>, true>(a, s);
    else
        launch_typed<Elem<AR_BF16>, false>(a, s);
    return hipGetLastError();
}

}  // namespace ar
