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
// Waves on a SIMD that its registers have to leave room for: 3 for bfloat16
// vectors of 16 bytes, where a fourth spills (8 ranks' 2048 x 10 bfloat16 heads of 128 by one
// workgroup a CU 66 us, by two 45, by three 37, when queries and keys still made
// their own angles).
template <class E, int W>
constexpr int back_waves()
{
    return W == 8 ? 3 : 2;
}

// A wave takes a run of one rank's tokens, a chunk of them at a time: cosines and
// sines for all its heads, in LDS of the wave's own, then the queries, 64 / lanes
// heads a round, then the keys.  Heads lie in registers as in the forward pass, the
// next round's loads in flight, and so do the wave's sums for the gradient of the
// side's weight (the other side's wait in LDS).  A workgroup's partial rows are
// added to the others' by k_heads_dw_join, in a fixed order.
//
// Bound by memory: 16384 x (16 + 4) bfloat16 heads of 256 move their 503 MB in 110
// us (4.6 TB/s), 8 ranks' 2048 x (8 + 2) of 128 their 126 MB in 34.
template <class E, int W, int LAYOUT, bool WHOLE>
__global__ __launch_bounds__(kThreads, (back_waves<E, W>())) void k_heads_back(HeadsBackArgs a)
{
    using H = Head<E, W, LAYOUT, WHOLE>;
    using T = typename E::T;
    extern __shared__ float4 s_all[];
    const uint32_t group = 64 / a.lanes, sub = (threadIdx.x & 63u) / a.lanes;
    const uint32_t lane = (threadIdx.x & 63u) - sub * a.lanes;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    touch(a);
    int one = a.heads[0] ? 0 : 1, two = a.heads[1] ? 1 : 0;  // first and last side there is
    // LDS: both weights (in registers they cost a wave on each SIMD), the waves' sums
    // of the side they are not at, their angles
    const HeadBackPlaces places = head_back_places(a.dim, kThreads, kThreads / 64, a.chunk * a.turn.pairs);
    float* s_w = reinterpret_cast<float*>(s_all);
    float4* s_acc = s_all + places.sums / 16 + threadIdx.x;
    float2* table = reinterpret_cast<float2*>(s_all) + places.angles / 8 +
                    wave * (a.chunk * a.turn.pairs);
    float acc[kHeadPerLane];
#pragma unroll
    for (int i = 0; i < kHeadPerLane; ++i)
        acc[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < kHeadPerLane / 4; ++i)
        s_acc[i * kThreads] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const auto change_sides = [&] {
#pragma unroll
        for (int i = 0; i < kHeadPerLane / 4; ++i) {
            const float4 o = s_acc[i * kThreads];
            s_acc[i * kThreads] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
            acc[4 * i] = o.x, acc[4 * i + 1] = o.y, acc[4 * i + 2] = o.z, acc[4 * i + 3] = o.w;
        }
    };

    // Where the wave is: a chunk (its batch, and its tokens there), a side, a round.
    // What a thread has of it: its head in the arrays, and that head's token in the
    // chunk.
    uint32_t number = blockIdx.x * (kThreads / 64) + wave;
    const bool apart = a.apart && one != two;  // a wave has one side of its (one) chunk
    const int from = one, to = two;
    if (apart) {
        one = two = number & 1u;
        number /= 2;
    }
    const uint32_t first = number * a.run;
    const uint32_t all = a.rank_batches * a.batch_chunks;
    const uint32_t end = first >= all ? 0 : all - first < a.run ? all : first + a.run;
    uint32_t b = 0, t0 = 0, count = 0;
    uint32_t h = 0, token = 0;
    const T *px = nullptr, *pdy = nullptr;
    T* pdx = nullptr;
    H x, dy;
    const auto load = [&] {
        dy.load(pdy, lane, a.lanes, a.nvec, a.turned);
        x.load(px, lane, a.lanes, a.nvec, a.turned);
    };
    const auto place = [&](uint32_t chunk) {
        const uint32_t in = divide(chunk, a.chunks);
        t0 = (chunk - in * a.batch_chunks) * a.chunk;
        count = a.tokens.by - t0 < a.chunk ? a.tokens.by - t0 : a.chunk;
        b = blockIdx.y * a.rank_batches + in;
    };
    // the first round of a side (a thread without a head: that of its last one)
    const auto enter = [&](int side) {
        const uint32_t rows = count * a.heads[side], row = sub < rows ? sub : rows - 1;
        token = divide(row, a.head[side]);
        h = row - token * a.heads[side];
        const auto at = [&](const HeadsArray& v) {
            return static_cast<T*>(v.p) + ((uint64_t)b * v.batch + (uint64_t)(t0 + token) * v.token +
                                           (uint64_t)h * v.head);
        };
        px = at(a.x[side]);
        pdy = at(a.dy[side]);
        pdx = at(a.dx[side]);
        load();
    };
    // dx of a head, and its part of dw
    float u[kHeadPerLane], n[kHeadPerLane];
    const auto head = [&](const float2* angles, int side) {
        if (a.turn.pairs)
            H::turn(u, angles, lane, a.lanes, a.turned, a.turn.pairs);
        const float r = head_rstd(n, a.lanes, a.dim, a.per_dim, a.eps);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kHeadPerLane; ++i) {
            n[i] *= r;
            acc[i] = fmaf(u[i], n[i], acc[i]);
        }
        const float* w = s_w + side * a.dim;
        H::each(lane, a.lanes, a.nvec, a.turned, [&](int i, uint32_t c) { u[i] *= w[c]; });
#pragma unroll
        for (int i = 0; i < kHeadPerLane; ++i)
            dot = fmaf(u[i], n[i], dot);
        const float m = lanes_total(dot, a.lanes) * a.per_dim;
#pragma unroll
        for (int i = 0; i < kHeadPerLane; ++i)
            u[i] = r * fmaf(-n[i], m, u[i]);
    };
    Weights<E> weights;
    weights.load(a.weight, a.weight_f32, a.dim);
    if (end) {
        place(first);
        enter(one);
    } else {
        count = 0;
    }
    // every wave makes a first turn, where it meets the others for the weights
    uint32_t chunk = first;
    do {
        if (a.turn.pairs)
            fill_angles(a.turn, a.tokens, b * a.tokens.by + t0, count, table);
        if (chunk == first) {
            weights.store(a.weight, a.weight_f32, a.dim, s_w);
            __syncthreads();
            if (!end)
                break;
        }
        const uint32_t tokens = count;
        for (int side = one; side <= two; ++side) {
            const HeadsStep s = a.step[side];
            const uint32_t heads = a.heads[side], rows = tokens * heads;
            uint32_t base = 0;
            for (; base + group < rows; base += group) {  // every thread has a head, and the wave another round
                const float2* angles = table + token * a.turn.pairs;
                T* out = pdx;
                dy.get(u, lane, a.lanes, a.nvec, a.turned);
                x.get(n, lane, a.lanes, a.nvec, a.turned);
                if (base + 2 * group <= rows || base + group + sub < rows) {
                    h += s.heads;
                    const bool wrap = h >= heads;
                    h -= wrap ? heads : 0;
                    token += s.tokens + wrap;
                    px += s.by[0] + (wrap ? s.more[0] : 0);
                    pdy += s.by[1] + (wrap ? s.more[1] : 0);
                    pdx += s.by[2] + (wrap ? s.more[2] : 0);
                }
                load();  // without another head: this one again
                head(angles, side);
                H::put(out, u, lane, a.lanes, a.nvec, a.turned, a.stream);
            }
            const float2* angles = table + token * a.turn.pairs;
            T* out = pdx;
            const bool on = base + sub < rows;
            if (!on) {
                // its sums get 0 * 1 / rms(1), whatever is, or by now was written, in what it read
                dy.set(0);
                x.set(sizeof(T) == 4 ? 0x3f800000u : 0x3f803f80u);
            }
            dy.get(u, lane, a.lanes, a.nvec, a.turned);
            x.get(n, lane, a.lanes, a.nvec, a.turned);
            if (side == two && chunk + 1 < end)
                place(chunk + 1);
            enter(side < two ? two : one);  // behind the last chunk: its first round again
            head(angles, side);
            if (on)
                H::put(out, u, lane, a.lanes, a.nvec, a.turned, a.stream);
            if (one != two)
                change_sides();
        }
    } while (++chunk < end);

    // the workgroup's sums: of the heads of a wave, then of the four waves
    float* s_dw = reinterpret_cast<float*>(s_all);
    float* p = a.partial + ((uint64_t)blockIdx.y * a.blocks + blockIdx.x) * 2 * a.dim;
    if (apart && one == 1)
        change_sides();
    float other[kHeadPerLane];
#pragma unroll
    for (int i = 0; i < kHeadPerLane / 4; ++i) {
        const float4 o = s_acc[i * kThreads];
        other[4 * i] = o.x, other[4 * i + 1] = o.y, other[4 * i + 2] = o.z, other[4 * i + 3] = o.w;
    }
    for (int side = from; side <= to; ++side) {
        for (uint32_t d = a.lanes; d < 64 && !(apart && side != one); d <<= 1)
#pragma unroll
            for (int i = 0; i < kHeadPerLane; ++i)
                acc[i] += __shfl_xor(acc[i], (int)d);
        __syncthreads();
        if ((threadIdx.x & 63u) < a.lanes)
            H::each(lane, a.lanes, a.nvec, a.turned,
                    [&](int i, uint32_t c) { s_dw[wave * a.dim + c] = acc[i]; });
        __syncthreads();
        for (uint32_t c = threadIdx.x; c < a.dim; c += kThreads)
            p[side * a.dim + c] = (s_dw[c] + s_dw[a.dim + c]) + (s_dw[2 * a.dim + c] + s_dw[3 * a.dim + c]);
#pragma unroll
        for (int i = 0; i < kHeadPerLane; ++i)
            acc[i] = other[i];
    }
}

// dweight[side][rank] = the sum of its partial rows (none: zeros): 32 columns to a
// workgroup, the rows dealt to 32 groups of threads (683 rows: 4.7 us, by 8 groups 7.8).
constexpr int kJoinCols = 32, kJoinGroups = 32;
struct Join {
    const float* partial;
    float* dweight[2];
    uint32_t blocks, dim;
};
__global__ __launch_bounds__(kJoinCols * kJoinGroups) void k_heads_dw_join(Join a)
{
    __shared__ float s_f[kJoinGroups][kJoinCols + 1];
    const uint32_t col = threadIdx.x % kJoinCols, g = threadIdx.x / kJoinCols;
    const uint32_t c = blockIdx.x * kJoinCols + col;
    const int side = blockIdx.z;
    float* dweight = side ? a.dweight[1] : a.dweight[0];
    if (!dweight)
        return;
    float acc = 0.0f;
    if (c < a.dim) {
        const float* p = a.partial + ((uint64_t)blockIdx.y * a.blocks * 2 + side) * a.dim + c;
#pragma unroll 8
        for (uint32_t b = g; b < a.blocks; b += kJoinGroups)
            acc += p[(uint64_t)b * 2 * a.dim];
    }
    s_f[g][col] = acc;
    __syncthreads();
    // 32 lanes a column, then: the groups' sums
    acc = lanes_sum(s_f[col][g], kJoinGroups);
    const uint32_t mine = blockIdx.x * kJoinCols + g;
    if (col == 0 && mine < a.dim)
        dweight[(uint64_t)blockIdx.y * a.dim + mine] = acc;
}

template <class E>
void launch_typed(int width, const HeadsBackArgs& a, size_t lds, hipStream_t s)
{
    const dim3 grid(a.blocks, a.ranks);
    with_width<E>(width, a.dim == a.lanes * kHeadPerLane, [&](auto w) {
        constexpr int W = decltype(w)::value;
        constexpr bool WHOLE = decltype(w)::whole;
        if (a.turn.layout == AR_ROTARY_HALVES)
            hipLaunchKernelGGL((k_heads_back<E, W, AR_ROTARY_HALVES, WHOLE>), grid, dim3(kThreads), lds, s,
                               a);
        else
            hipLaunchKernelGGL((k_heads_back<E, W, AR_ROTARY_PAIRS, WHOLE>), grid, dim3(kThreads), lds, s,
                               a);
    });
}

}  // namespace

hipError_t launch_heads_back(int dtype, HeadsBackArgs a, hipStream_t s)
{
    const int w = heads_vector(dtype, a.dim, a.turn);
    heads_fit(a.dim, w, &a.nvec, &a.turned, &a.lanes, &a.turn);
    const uint32_t group = 64 / a.lanes, waves = kThreads / 64;
    const uint64_t all = (uint64_t)a.rank_tokens * (a.heads[0] + a.heads[1]) * a.ranks;
    a.stream = all * a.dim * (dtype == AR_BF16 ? 2 : 4) > kStreamBytes;
    a.per_dim = 1.0f / (float)a.dim;
    a.blocks = 0;
    if (a.rank_tokens) {
        for (int side = 0; side < 2; ++side) {
            HeadsStep& step = a.step[side];
            const uint32_t heads = a.heads[side];
            if (!heads)
                continue;
            step.heads = group % heads;
            step.tokens = group / heads;
            const HeadsArray* const arrays[3] = {&a.x[side], &a.dy[side], &a.dx[side]};
            for (int i = 0; i < 3; ++i) {
                const HeadsArray& v = *arrays[i];
                step.by[i] = step.tokens * v.token + step.heads * v.head;
                step.more[i] = v.token - heads * v.head;
            }
        }
        // tokens whose heads of both sides fill rounds (8 ranks' 2048 x (8 + 2) heads of
        // 128: 4), fewer while the chip has not enough; fewer still, and waves have one
        // side each (2 x 333 x (6 + 6) float32 heads of 96: 9.9 us, 11.5 before)
        a.chunk = group;
        while (a.chunk > 1 && a.chunk / 2 * a.heads[0] % group == 0 && a.chunk / 2 * a.heads[1] % group == 0)
            a.chunk /= 2;
        const uint32_t most = (uint32_t)head_back_blocks(a.ranks);
        while (a.chunk > 1 && (uint64_t)a.rank_tokens < (uint64_t)a.chunk * most * waves)
            a.chunk /= 2;
        a.batch_chunks = (a.tokens.by + a.chunk - 1) / a.chunk;
        a.chunks = fast_div(a.batch_chunks);
        const uint32_t chunks = a.batch_chunks * a.rank_batches;
        a.apart = a.heads[0] && a.heads[1] && 2 * (uint64_t)chunks <= most * waves;
        const uint32_t units = a.apart ? 2 * chunks : chunks;
        a.run = (units + most * waves - 1) / (most * waves);
        a.blocks = (units + a.run * waves - 1) / (a.run * waves);
        const size_t lds = head_back_places(a.dim, kThreads, waves, a.chunk * a.turn.pairs).bytes;
        if (dtype == AR_FLOAT32)
            launch_typed<Elem<AR_FLOAT32>>(w, a, lds, s);
        else
            launch_typed<Elem<AR_BF16>>(w, a, lds, s);
    }
    hipLaunchKernelGGL(k_heads_dw_join, dim3((a.dim + kJoinCols - 1) / kJoinCols, a.ranks, 2),
                       dim3(kJoinCols * kJoinGroups), 0, s,
                       Join{a.partial, {a.dweight[0], a.dweight[1]}, a.blocks, a.dim});
    return hipGetLastError();
}

}  // namespace ar
