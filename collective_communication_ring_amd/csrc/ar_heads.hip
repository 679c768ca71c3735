// ar_heads.hip -- position rotation of attention heads, alone or behind an RMS
// norm of each head.
//
//   r = 1 / sqrt(mean(x^2) + eps),  v = x r w      (norm only; else v = x)
//   (a, b) -> (c a - s b, c b + s a)  for each pair of v's first rot_dim
#include <algorithm>

#include "ar_heads_common.h"

namespace ar {
namespace {

constexpr int kThreads = 256;

// A head lies in the registers of `lanes` threads, 16 elements each, two vectors
// of a pair in one thread in both layouts, so the rotation needs no exchange.  A
// wave takes `turns` rounds of 64 / lanes heads, of queries and keys alike, token
// by token, the next round's loads in flight; it computes cosines and sines once
// for each of its tokens, into LDS of its own.
//
// Bound by memory: 16384 x (32 + 8) bfloat16 heads of 128 are rotated, 335 MB moved,
// in 62 us (5.4 TB/s), 8 ranks' 2048 x (8 + 2) normed and rotated, 84 MB, in 18.
template <class E, int W, bool NORM, int LAYOUT, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_heads(HeadsArgs a)
{
    using H = Head<E, W, LAYOUT, WHOLE>;
    using T = typename E::T;
    extern __shared__ float2 s_table[];
    const uint32_t group = 64 / a.lanes, sub = (threadIdx.x & 63u) / a.lanes;
    const uint32_t lane = (threadIdx.x & 63u) - sub * a.lanes;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t row0 = ((a.first + blockIdx.x) * (kThreads / 64) + wave) * (group * a.turns);
    const uint32_t rows = row0 >= a.rows ? 0 : a.rows - row0 < group * a.turns ? a.rows - row0
                                                                              : group * a.turns;
    struct At {
        uint32_t token, side, b, t, h;
    };
    const auto place = [&](uint32_t k) {
        const uint32_t i = k * group + sub;
        // no thread without a head: the last one there is
        const uint32_t row = i < rows ? row0 + i : rows ? row0 + rows - 1 : a.rows - 1;
        At o;
        o.token = divide(row, a.heads);
        o.h = row - o.token * a.heads.by;
        o.side = o.h >= a.heads0;
        o.h -= o.side ? a.heads0 : 0;
        o.b = divide(o.token, a.tokens);
        o.t = o.token - o.b * a.tokens.by;
        return o;
    };
    const auto address = [&](const HeadsArray (&x)[2], const At& o) {
        const HeadsArray v = o.side ? x[1] : x[0];
        return static_cast<T*>(v.p) + (o.b * v.batch + o.t * v.token + o.h * v.head);
    };

    H cur;
    At at = place(0);
    cur.load(address(a.x, at), lane, a.lanes, a.nvec, a.turned);
    float* s_w = reinterpret_cast<float*>(s_table);
    float2* table = s_table + wave * a.table;
    Weights<E> weights;
    if constexpr (NORM) {
        table += a.dim;  // behind both weights
        weights.load(a.weight, a.weight_f32, a.dim);
    }
    const uint32_t first = divide(row0, a.heads);
    if (rows && a.turn.pairs)
        fill_angles(a.turn, a.tokens, first, divide(row0 + rows - 1, a.heads) - first + 1, table);
    if constexpr (NORM) {
        weights.store(a.weight, a.weight_f32, a.dim, s_w);
        __syncthreads();
    }
    if (!rows)
        return;
    const auto head = [&](const At& here, float (&v)[kHeadPerLane]) {
        if constexpr (NORM) {
            const float r = head_rstd(v, a.lanes, a.dim, a.per_dim, a.eps);
            const float* w = s_w + (here.side ? a.dim : 0);
            H::each(lane, a.lanes, a.nvec, a.turned, [&](int i, uint32_t c) { v[i] = v[i] * r * w[c]; });
        }
        if (a.turn.pairs)
            H::turn(v, table + (here.token - first) * a.turn.pairs, lane, a.lanes, a.turned, a.turn.pairs);
    };
    float v[kHeadPerLane];
    uint32_t k = 0;
    for (; (k + 1) * group < rows; ++k) {  // every thread has a head, and the wave another round
        const At here = at;
        cur.get(v, lane, a.lanes, a.nvec, a.turned);
        at = place(k + 1);
        cur.load(address(a.x, at), lane, a.lanes, a.nvec, a.turned);
        head(here, v);
        H::put(address(a.y, here), v, lane, a.lanes, a.nvec, a.turned, a.stream);
    }
    cur.get(v, lane, a.lanes, a.nvec, a.turned);
    head(at, v);
    if (k * group + sub < rows)
        H::put(address(a.y, at), v, lane, a.lanes, a.nvec, a.turned, a.stream);
}

template <class E, bool NORM>
void launch_typed(int width, const HeadsArgs& a, size_t lds, uint32_t grid, hipStream_t s)
{
    with_width<E>(width, a.dim == a.lanes * kHeadPerLane, [&](auto w) {
        constexpr int W = decltype(w)::value;
        constexpr bool WHOLE = decltype(w)::whole;
        if (a.turn.layout == AR_ROTARY_HALVES)
            hipLaunchKernelGGL((k_heads<E, W, NORM, AR_ROTARY_HALVES, WHOLE>), dim3(grid), dim3(kThreads),
                               lds, s, a);
        else
            hipLaunchKernelGGL((k_heads<E, W, NORM, AR_ROTARY_PAIRS, WHOLE>), dim3(grid), dim3(kThreads),
                               lds, s, a);
    });
}

}  // namespace

int heads_vector(int dtype, uint32_t dim, const Turn& t)
{
    int w = dtype == AR_BF16 ? 8 : 4;
    while (w > 1 && (dim % w || (t.layout == AR_ROTARY_HALVES && t.pairs % w)))
        w /= 2;
    return w;
}

// The last fields of the arguments, for vectors of `w` elements.
void heads_fit(uint32_t dim, int w, uint32_t* nvec, uint32_t* turned, uint32_t* lanes, Turn* t)
{
    *nvec = dim / w;
    *turned = t->layout == AR_ROTARY_HALVES ? t->pairs / w : 0;
    for (t->lanes = 1; t->lanes < 64 && t->lanes < t->pairs;)
        t->lanes *= 2;
    *lanes = 1;
    while (*lanes * kHeadPerLane < dim)
        *lanes *= 2;
}

hipError_t launch_heads(int dtype, bool norm, HeadsArgs a, hipStream_t s)
{
    const int w = heads_vector(dtype, a.dim, a.turn);
    heads_fit(a.dim, w, &a.nvec, &a.turned, &a.lanes, &a.turn);
    a.per_dim = 1.0f / (float)a.dim;
    a.stream = (uint64_t)a.rows * a.dim * (dtype == AR_BF16 ? 2 : 4) > kStreamBytes;
    const uint32_t group = 64 / a.lanes, waves = kThreads / 64;
    const auto table = [&](uint32_t turns) {  // cosines and sines of a wave's tokens
        const uint32_t n = group * turns;  // whole tokens, or it may begin within one
        return (n % a.heads.by ? (n + a.heads.by - 2) / a.heads.by + 1 : n / a.heads.by) * a.turn.pairs;
    };
    // Rounds of a wave: those of whole tokens, 4 at least, where enough waves are left
    // to fill the chip (8 ranks' 2048 x 10 heads of 128: 19.9 us by 4 or 5 rounds, 22.1
    // by 2, 25.0 by one, 23.0 by 10), else as many as leave enough.
    const uint32_t rounds = (a.rows + group - 1) / group;
    uint32_t tokens = group;  // whose heads fill rounds: group / gcd(group, heads), a power of two
    while (tokens > 1 && tokens / 2 * a.heads.by % group == 0)
        tokens /= 2;
    const uint32_t whole = tokens * a.heads.by / group;
    a.turns = whole < 4 ? (3 + whole) / whole * whole : whole;
    if (a.turns > 8 || rounds / a.turns < 4096)
        a.turns = std::max(1u, std::min(4u, rounds / 4096));
    while (a.turns > 1 && table(a.turns) > 1024)
        --a.turns;
    a.table = table(a.turns);
    const size_t lds = waves * a.table * sizeof(float2) + (norm ? 8 * (size_t)a.dim : 0);
    const uint32_t blocks = (rounds + a.turns * waves - 1) / (a.turns * waves);
    a.first = 0;
    for (; a.first < blocks; a.first += kHeadsMostBlocks) {
        const uint32_t grid = std::min(blocks - a.first, kHeadsMostBlocks);
        if (dtype == AR_FLOAT32)
            norm ? launch_typed<Elem<AR_FLOAT32>, true>(w, a, lds, grid, s)
                 : launch_typed<Elem<AR_FLOAT32>, false>(w, a, lds, grid, s);
        else
            norm ? launch_typed<Elem<AR_BF16>, true>(w, a, lds, grid, s)
                 : launch_typed<Elem<AR_BF16>, false>(w, a, lds, grid, s);
    }
    return hipGetLastError();
}

}  // namespace ar
