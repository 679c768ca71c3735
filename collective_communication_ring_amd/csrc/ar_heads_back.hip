// ar_heads_back.hip -- backward pass of the head norm with its rotation.
//
//   u = rotation^T dy,  n = x r,  g = u w:
//   dx = r (g - n mean(g n)),   dw = sum over heads of u n
//
// r is taken again from x, which is read anyway: nothing but x is kept from
// the forward pass.
#include <algorithm>

#include "ar_heads_common.h"

namespace ar {
namespace {

constexpr int kThreads = 256;

// A workgroup takes heads of one side (queries or keys) of one rank, 256 /
// lanes at a time, and keeps its sums for dw in registers; heads lie in
// registers as in the forward pass.  Its partial row is added to the others'
// by k_heads_dw_join, in a fixed order.
template <class E, int W, bool NT>
__global__ __launch_bounds__(kThreads) void k_heads_back(HeadsBackArgs a)
{
    using H = Head<E, W>;
    using T = typename E::T;
    extern __shared__ float2 s_table[];
    const uint32_t group = kThreads / a.lanes, sub = threadIdx.x / a.lanes;
    const uint32_t lane = threadIdx.x - sub * a.lanes;
    const int side = blockIdx.x >= (uint32_t)a.blocks[0];
    const uint32_t block = blockIdx.x - (side ? a.blocks[0] : 0), blocks = a.blocks[side];
    const uint32_t rows = a.rows[side], token0 = blockIdx.y * a.rank_tokens;
    const HeadsArray DY = a.dy[side], X = a.x[side], DX = a.dx[side];
    const FastDiv heads = a.head[side];
    const int layout = a.turn.layout;
    float acc[kHeadPerLane], w[kHeadPerLane];
#pragma unroll
    for (int i = 0; i < kHeadPerLane; ++i)
        acc[i] = w[i] = 0.0f;
    H::each(lane, a.lanes, a.nvec, a.turned, layout,
            [&](int i, uint32_t c) { w[i] = weight_at<E>(a.weight[side], a.weight_f32, c); });

    // every thread makes every turn, also one without a head: they meet at barriers
    for (uint32_t base = block * group; base < rows; base += blocks * group) {
        const bool on = base + sub < rows;
        const uint32_t row = on ? base + sub : rows - 1;
        const uint32_t token = divide(row, heads), h = row - token * heads.by;
        const uint32_t all = token0 + token, b = divide(all, a.tokens), t = all - b * a.tokens.by;
        H x, dy;
        dy.load(static_cast<const T*>(DY.p) + (b * DY.batch + t * DY.token + h * DY.head), lane,
                a.lanes, a.nvec, a.turned, layout);
        x.load(static_cast<const T*>(X.p) + (b * X.batch + t * X.token + h * X.head), lane, a.lanes,
               a.nvec, a.turned, layout);
        const uint32_t first = divide(base, heads);
        if (a.turned) {
            const uint32_t last = base + group < rows ? base + group - 1 : rows - 1;
            __syncthreads();
            fill_angles(a.turn, a.tokens, token0 + first, divide(last, heads) - first + 1,
                        token0 + a.rank_tokens, s_table);
            __syncthreads();
        }
        float u[kHeadPerLane], n[kHeadPerLane];
        dy.get(u, lane, a.lanes, a.nvec, a.turned, layout);
        x.get(n, lane, a.lanes, a.nvec, a.turned, layout);
        if (a.turned)
            H::turn(u, s_table + (token - first) * a.turn.slots, lane, a.lanes, a.turned,
                    a.turn.pairs, layout);
        const float r = head_rstd(n, a.lanes, a.dim, a.eps);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kHeadPerLane; ++i) {
            n[i] *= r;
            acc[i] = fmaf(on ? u[i] : 0.0f, on ? n[i] : 0.0f, acc[i]);
            u[i] *= w[i];
            dot = fmaf(u[i], n[i], dot);
        }
        const float m = lanes_total(dot, a.lanes) / (float)a.dim;
#pragma unroll
        for (int i = 0; i < kHeadPerLane; ++i)
            u[i] = r * (u[i] - n[i] * m);
        if (on)
            H::template put<NT>(static_cast<T*>(DX.p) + (b * DX.batch + t * DX.token + h * DX.head),
                                u, lane, a.lanes, a.nvec, a.turned, layout);
    }

    // the workgroup's heads: those of a wave, then the four waves'
    for (uint32_t d = a.lanes; d < 64; d <<= 1)
#pragma unroll
        for (int i = 0; i < kHeadPerLane; ++i)
            acc[i] += __shfl_xor(acc[i], (int)d);
    float* s_dw = reinterpret_cast<float*>(s_table);
    __syncthreads();
    const uint32_t wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63u) < a.lanes)
        H::each(lane, a.lanes, a.nvec, a.turned, layout,
                [&](int i, uint32_t c) { s_dw[wave * a.dim + c] = acc[i]; });
    __syncthreads();
    float* p = a.partial +
               ((uint64_t)blockIdx.y * (a.blocks[0] + a.blocks[1]) + blockIdx.x) * a.dim;
    for (uint32_t c = threadIdx.x; c < a.dim; c += kThreads)
        p[c] = (s_dw[c] + s_dw[a.dim + c]) + (s_dw[2 * a.dim + c] + s_dw[3 * a.dim + c]);
}

// dweight[side][rank] = the sum of its partial rows (none: zeros): 32 columns
// to a workgroup, the rows dealt to 8 groups of threads.
constexpr int kJoinCols = 32;
__global__ __launch_bounds__(kThreads) void k_heads_dw_join(HeadsBackArgs a)
{
    constexpr int G = kThreads / kJoinCols;
    __shared__ float s_f[G][kJoinCols];
    const uint32_t col = threadIdx.x % kJoinCols, g = threadIdx.x / kJoinCols;
    const uint32_t c = blockIdx.x * kJoinCols + col;
    const int side = blockIdx.z;
    if (!a.dweight[side])
        return;
    float acc = 0.0f;
    if (c < a.dim) {
        const uint64_t row = (uint64_t)blockIdx.y * (a.blocks[0] + a.blocks[1]) +
                             (side ? a.blocks[0] : 0);
        const float* p = a.partial + row * a.dim + c;
#pragma unroll 8
        for (int b = g; b < a.blocks[side]; b += G)
            acc += p[(uint64_t)b * a.dim];
    }
    s_f[g][col] = acc;
    __syncthreads();
    if (g || c >= a.dim)
        return;
#pragma unroll
    for (int o = 1; o < G; ++o)
        acc += s_f[o][col];
    a.dweight[side][(uint64_t)blockIdx.y * a.dim + c] = acc;
}

template <class E, int W>
void launch_width(const HeadsBackArgs& a, size_t lds, hipStream_t s)
{
    const dim3 grid(a.blocks[0] + a.blocks[1], a.ranks);
    if (a.stream)
        hipLaunchKernelGGL((k_heads_back<E, W, true>), grid, dim3(kThreads), lds, s, a);
    else
        hipLaunchKernelGGL((k_heads_back<E, W, false>), grid, dim3(kThreads), lds, s, a);
}

template <class E>
void launch_typed(int width, const HeadsBackArgs& a, size_t lds, hipStream_t s)
{
    if constexpr (E::VEC == 8)
        if (width == 8)
            return launch_width<E, 8>(a, lds, s);
    if (width == 4)
        launch_width<E, 4>(a, lds, s);
    else if (width == 2)
        launch_width<E, 2>(a, lds, s);
    else
        launch_width<E, 1>(a, lds, s);
}

}  // namespace

hipError_t launch_heads_back(int dtype, HeadsBackArgs a, hipStream_t s)
{
    const int w = heads_vector(dtype, a.dim, a.turn);
    heads_fit(a.dim, w, &a.nvec, &a.turned, &a.lanes, &a.turn);
    const uint32_t group = kThreads / a.lanes;
    const uint64_t all = ((uint64_t)a.rows[0] + a.rows[1]) * a.ranks;
    a.stream = all * a.dim * (dtype == AR_BF16 ? 2 : 4) > kStreamBytes;
    // workgroups to each side by its share of the heads
    const int total = head_back_blocks(a.ranks);
    size_t lds = 4 * sizeof(float) * a.dim;
    for (int side = 0; side < 2; ++side) {
        a.blocks[side] = 0;
        if (!a.rows[side])
            continue;
        const uint32_t rounds = (a.rows[side] + group - 1) / group;
        const uint64_t part = (uint64_t)total * a.heads[side] / (a.heads[0] + a.heads[1]);
        const uint64_t most = std::max<uint64_t>(1, a.rows[!side] ? std::min<uint64_t>(part, total - 1)
                                                                  : total);
        a.blocks[side] = (int)std::min<uint64_t>(rounds, most);
        const uint32_t tokens = (group + a.heads[side] - 2) / a.heads[side] + 1;
        lds = std::max(lds, (size_t)tokens * a.turn.slots * sizeof(float2));
    }
    if (a.blocks[0] + a.blocks[1]) {
        if (dtype == AR_FLOAT32)
            launch_typed<Elem<AR_FLOAT32>>(w, a, lds, s);
        else
            launch_typed<Elem<AR_BF16>>(w, a, lds, s);
    }
    hipLaunchKernelGGL(k_heads_dw_join, dim3((a.dim + kJoinCols - 1) / kJoinCols, a.ranks, 2),
                       dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace ar
