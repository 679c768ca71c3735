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

// A head lies in the registers of `lanes` threads, 16 elements each, two
// vectors of a pair in one thread in both layouts, so the rotation needs no
// exchange.  A workgroup takes `turns` rounds of 256 / lanes heads, of queries
// and keys alike, token by token; cosines and sines are computed once for each
// of its tokens, into LDS, while the first heads' loads are in flight.
template <class E, int W, bool NORM, bool NT>
__global__ __launch_bounds__(kThreads) void k_heads(HeadsArgs a)
{
    using H = Head<E, W>;
    using T = typename E::T;
    extern __shared__ float2 s_table[];
    const uint32_t group = kThreads / a.lanes, sub = threadIdx.x / a.lanes;
    const uint32_t lane = threadIdx.x - sub * a.lanes;
    const uint32_t row0 = blockIdx.x * (group * a.turns);
    const uint32_t rows = a.rows - row0 < group * a.turns ? a.rows - row0 : group * a.turns;
    const uint32_t first = divide(row0, a.heads);
    const uint32_t count = divide(row0 + rows - 1, a.heads) - first + 1;
    const uint32_t end = divide(a.rows - 1, a.heads) + 1;
    const int layout = a.turn.layout;

    struct At {
        uint32_t token, side, b, t, h;
    };
    const auto place = [&](uint32_t k) {
        const uint32_t i = k * group + sub;
        const uint32_t row = row0 + (i < rows ? i : rows - 1);  // no thread without a head
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
    cur.load(address(a.x, at), lane, a.lanes, a.nvec, a.turned, layout);
    float* s_w = reinterpret_cast<float*>(s_table);
    float2* table = s_table;
    if constexpr (NORM) {
        table += a.dim;  // behind both weights
        for (uint32_t c = threadIdx.x; c < a.dim; c += kThreads) {
            s_w[c] = a.weight[0] ? weight_at<E>(a.weight[0], a.weight_f32, c) : 0.0f;
            s_w[a.dim + c] = a.weight[1] ? weight_at<E>(a.weight[1], a.weight_f32, c) : 0.0f;
        }
    }
    if (a.turned)
        fill_angles(a.turn, a.tokens, first, count, end, table);
    __syncthreads();
    for (uint32_t k = 0; k < a.turns && k * group < rows; ++k) {
        const At here = at;
        float v[kHeadPerLane];
        cur.get(v, lane, a.lanes, a.nvec, a.turned, layout);
        if (k + 1 < a.turns) {
            at = place(k + 1);
            cur.load(address(a.x, at), lane, a.lanes, a.nvec, a.turned, layout);
        }
        if constexpr (NORM) {
            const float r = head_rstd(v, a.lanes, a.dim, a.eps);
            const float* w = s_w + (here.side ? a.dim : 0);
            H::each(lane, a.lanes, a.nvec, a.turned, layout,
                    [&](int i, uint32_t c) { v[i] = v[i] * r * w[c]; });
        }
        if (a.turned)
            H::turn(v, table + (here.token - first) * a.turn.slots, lane, a.lanes, a.turned,
                    a.turn.pairs, layout);
        if (k * group + sub < rows)
            H::template put<NT>(address(a.y, here), v, lane, a.lanes, a.nvec, a.turned, layout);
    }
}

template <class E, int W, bool NORM>
void launch_width(const HeadsArgs& a, size_t lds, uint32_t grid, hipStream_t s)
{
    if (a.stream)
        hipLaunchKernelGGL((k_heads<E, W, NORM, true>), dim3(grid), dim3(kThreads), lds, s, a);
    else
        hipLaunchKernelGGL((k_heads<E, W, NORM, false>), dim3(grid), dim3(kThreads), lds, s, a);
}

template <class E, bool NORM>
void launch_typed(int width, const HeadsArgs& a, size_t lds, uint32_t grid, hipStream_t s)
{
    if constexpr (E::VEC == 8)
        if (width == 8)
            return launch_width<E, 8, NORM>(a, lds, grid, s);
    if (width == 4)
        launch_width<E, 4, NORM>(a, lds, grid, s);
    else if (width == 2)
        launch_width<E, 2, NORM>(a, lds, grid, s);
    else
        launch_width<E, 1, NORM>(a, lds, grid, s);
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
    *turned = (t->pairs + w - 1) / w;
    t->slots = *turned * w;
    t->per_slot = fast_div(t->slots ? t->slots : 1);
    *lanes = 1;
    while (*lanes * kHeadPerLane < dim)
        *lanes *= 2;
}

hipError_t launch_heads(int dtype, bool norm, HeadsArgs a, hipStream_t s)
{
    const int w = heads_vector(dtype, a.dim, a.turn);
    heads_fit(a.dim, w, &a.nvec, &a.turned, &a.lanes, &a.turn);
    a.stream = (uint64_t)a.rows * a.dim * (dtype == AR_BF16 ? 2 : 4) > kStreamBytes;
    const uint32_t group = kThreads / a.lanes;
    const auto lds = [&](uint32_t turns) {
        const uint32_t n = group * turns, tokens = (n + a.heads.by - 2) / a.heads.by + 1;
        return (size_t)tokens * a.turn.slots * sizeof(float2) + (norm ? 8 * (size_t)a.dim : 0);
    };
    const uint32_t rounds = (a.rows + group - 1) / group;
    a.turns = std::max(1u, std::min(4u, rounds / 2048));
    while (a.turns > 1 && lds(a.turns) > 20480)
        --a.turns;
    const uint32_t grid = (rounds + a.turns - 1) / a.turns;
    if (dtype == AR_FLOAT32)
        norm ? launch_typed<Elem<AR_FLOAT32>, true>(w, a, lds(a.turns), grid, s)
             : launch_typed<Elem<AR_FLOAT32>, false>(w, a, lds(a.turns), grid, s);
    else
        norm ? launch_typed<Elem<AR_BF16>, true>(w, a, lds(a.turns), grid, s)
             : launch_typed<Elem<AR_BF16>, false>(w, a, lds(a.turns), grid, s);
    return hipGetLastError();
}

}  // namespace ar
