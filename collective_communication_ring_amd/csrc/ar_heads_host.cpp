// ar_heads_host.cpp -- host side of the operators on attention heads: argument
// checks, overlaps of strided arrays, and rotary frequencies.
#include <algorithm>
#include <cmath>

#include "ar_checks.h"
#include "ar_heads.h"

using namespace ar;

namespace {

constexpr uint64_t kMaxHeads = ((uint64_t)1 << 31) - 1;  // of a call, batches and tokens included

// An array as nested repetitions of a block of bytes, smallest distance first;
// those of one, and those that only continue the block, are left out.
struct Nest {
    uintptr_t at = 0;
    uint64_t len = 0;  // 0: no bytes
    int levels = 0;
    uint64_t n[3], step[3];
    uint64_t apart[3] = {0, 0, 0};  // heads, tokens and batches as they are (of one: 0)
};

// Bytes that the first `levels` levels span.
uint64_t span(const Nest& a, int levels)
{
    uint64_t s = a.len;
    for (int i = 0; i < levels; ++i)
        s += (a.n[i] - 1) * a.step[i];
    return s;
}

// The nest of an array of heads; false: distances too large, or not nested
// (then the array has an element twice, or is taken to).
bool nest_of(const ar_heads_t& h, uint64_t batch, uint64_t tokens, uint64_t heads, uint64_t dim,
             size_t z, Nest* out, bool* nested)
{
    struct Level {
        uint64_t n, step;
    } l[3] = {{heads, h.head_stride}, {tokens, h.token_stride}, {batch, h.batch_stride}};
    for (const Level& v : l)
        if (v.n > 1 && v.step > kMaxElems / (v.n - 1))
            return false;
    std::sort(l, l + 3, [](const Level& a, const Level& b) {
        return a.n == 1 || b.n == 1 ? a.n == 1 && b.n != 1 : a.step < b.step;
    });
    *out = Nest{};
    out->at = (uintptr_t)h.data;
    out->len = dim * z;
    out->apart[0] = heads > 1 ? h.head_stride : 0;
    out->apart[1] = tokens > 1 ? h.token_stride : 0;
    out->apart[2] = batch > 1 ? h.batch_stride : 0;
    *nested = true;
    for (const Level& v : l) {
        if (v.n == 1)
            continue;
        const uint64_t step = v.step * z;
        if (step < span(*out, out->levels))
            *nested = false;
        if (!step)
            continue;  // the same bytes again
        if (out->levels == 0 && step == out->len) {
            out->len *= v.n;
        } else if (out->levels && step == out->n[out->levels - 1] * out->step[out->levels - 1]) {
            out->n[out->levels - 1] *= v.n;
        } else {
            out->n[out->levels] = v.n;
            out->step[out->levels++] = step;
        }
    }
    return true;
}

// Whether the first `la` levels of a, at address x, and the first `lb` of b, at
// y, may share a byte.  Exact where the levels have the same distances: blocks
// that lie in turn then miss each other.
bool share(const Nest& a, int la, uintptr_t x, const Nest& b, int lb, uintptr_t y)
{
    const uint64_t sa = span(a, la), sb = span(b, lb);
    if (x + sa <= y || y + sb <= x)
        return false;
    if (!la && !lb)
        return true;
    const uint64_t step = !la ? b.step[lb - 1] : a.step[la - 1];
    // one that is a single block, or repeats further apart, is met by any of the
    // other's repetitions as if it were one of its own distance
    if (la && lb && a.step[la - 1] != b.step[lb - 1])
        return true;
    const int ia = la ? la - 1 : 0, ib = lb ? lb - 1 : 0;
    const uint64_t ea = span(a, ia), eb = span(b, ib);
    if (ea > step || eb > step)
        return true;
    const uint64_t d = y >= x ? (y - x) % step : (step - (x - y) % step) % step;
    // b's block begins d behind one of a's, and step - d ahead of the next
    const uintptr_t base = (uintptr_t)1 << 60;
    return share(a, ia, base, b, ib, base + d) || share(a, ia, base + step, b, ib, base + d);
}

bool share(const Nest& a, const Nest& b)
{
    return a.len && b.len && share(a, a.levels, a.at, b, b.levels, b.at);
}

// Every element at the same address (of arrays with the same sizes).
bool same(const Nest& a, const Nest& b)
{
    return a.at == b.at && std::equal(a.apart, a.apart + 3, b.apart);
}

Nest block(const void* p, uint64_t bytes)
{
    Nest n;
    n.at = (uintptr_t)p;
    n.len = p ? bytes : 0;
    return n;
}

// Arrays of one call, outputs first.  own[i]: which inputs output i may replace.
struct Arrays {
    Nest out[8], in[12];
    unsigned own[8];
    int nout = 0, nin = 0;
};

bool disjoint(const Arrays& a)
{
    for (int i = 0; i < a.nout; ++i) {
        for (int j = i + 1; j < a.nout; ++j)
            if (share(a.out[i], a.out[j]))
                return false;
        for (int j = 0; j < a.nin; ++j)
            if (share(a.out[i], a.in[j]) && !(a.own[i] >> j & 1 && same(a.out[i], a.in[j])))
                return false;
    }
    return true;
}

struct Shape {
    int dtype;
    size_t batch, tokens, heads[2], dim;
};

// Sizes that no call has, and those that do nothing.
int check_shape(const Shape& s, bool* nothing)
{
    if (!stream_type(s.dtype) || s.dim < 1 || s.dim > kHeadMaxDim)
        return AR_ERR_INVALID_ARG;
    for (size_t n : {s.batch, s.tokens, s.heads[0], s.heads[1]})
        if (n > kMaxHeads)
            return AR_ERR_INVALID_ARG;
    const uint64_t tokens = (uint64_t)s.batch * s.tokens, heads = (uint64_t)s.heads[0] + s.heads[1];
    *nothing = !tokens || !heads;
    if (!*nothing && tokens > kMaxHeads / heads)
        return AR_ERR_INVALID_ARG;
    return AR_SUCCESS;
}

// Adds an array of heads to a call's (side: queries or keys).
int add_heads(const Shape& s, int side, const ar_heads_t& h, bool output, unsigned own, Arrays* all)
{
    if (!s.heads[side]) {  // holds its place
        if (output) {
            all->own[all->nout] = 0;
            all->out[all->nout++] = Nest{};
        } else {
            all->in[all->nin++] = Nest{};
        }
        return AR_SUCCESS;
    }
    Nest n;
    bool nested = false;
    if (!h.data || misaligned(h.data, s.dtype) ||
        !nest_of(h, s.batch, s.tokens, s.heads[side], s.dim, size_of(s.dtype), &n, &nested))
        return AR_ERR_INVALID_ARG;
    if (output) {
        if (!nested)
            return AR_ERR_INVALID_ARG;
        all->own[all->nout] = own;
        all->out[all->nout++] = n;
    } else {
        all->in[all->nin++] = n;
    }
    return AR_SUCCESS;
}

// The rotation's checks, arrays and kernel form.
int add_turn(const Shape& s, const ar_rotation_t& r, bool inverse, Arrays* all, Turn* out)
{
    *out = Turn{};
    if (r.rot_dim > s.dim || r.rot_dim % 2)
        return AR_ERR_INVALID_ARG;
    out->layout = AR_ROTARY_PAIRS;
    if (!r.rot_dim)
        return AR_SUCCESS;
    if ((r.layout != AR_ROTARY_HALVES && r.layout != AR_ROTARY_PAIRS) || !std::isfinite(r.factor) ||
        (r.position_bytes != 4 && r.position_bytes != 8) || !r.frequencies || !r.positions ||
        (uintptr_t)r.frequencies % 8 || (uintptr_t)r.positions % (uintptr_t)r.position_bytes)
        return AR_ERR_INVALID_ARG;
    if (s.batch > 1 && r.position_stride > kMaxElems / (s.batch - 1))
        return AR_ERR_INVALID_ARG;
    out->frequencies = r.frequencies;
    out->positions = r.positions;
    out->position_stride = s.batch > 1 ? r.position_stride : 0;
    out->wide = r.position_bytes == 8;
    out->layout = r.layout;
    out->pairs = (uint32_t)(r.rot_dim / 2);
    out->factor = r.factor;
    out->sign = inverse ? -1.0f : 1.0f;
    all->in[all->nin++] = block(r.frequencies, r.rot_dim / 2 * 8);
    all->in[all->nin++] = block(
        r.positions, ((s.batch - 1) * out->position_stride + s.tokens) * (size_t)r.position_bytes);
    return AR_SUCCESS;
}

int add_weights(const Shape& s, int weight_dtype, const void* const (&w)[2], Arrays* all)
{
    if (weight_dtype != s.dtype && weight_dtype != AR_FLOAT32)
        return AR_ERR_INVALID_ARG;
    for (int side = 0; side < 2; ++side) {
        if (!s.heads[side])
            continue;
        if (!w[side] || misaligned(w[side], weight_dtype))
            return AR_ERR_INVALID_ARG;
        all->in[all->nin++] = block(w[side], s.dim * size_of(weight_dtype));
    }
    return AR_SUCCESS;
}

bool bad_eps(float eps) { return !(eps >= 0.0f) || std::isinf(eps); }

HeadsArray array_of(const ar_heads_t& h)
{
    return {h.data, h.batch_stride, h.token_stride, h.head_stride};
}

#define TRY(call)                  \
    do {                           \
        const int rc_ = (call);    \
        if (rc_ != AR_SUCCESS)     \
            return rc_;            \
    } while (0)

// The forward operators: everything but the launch.
int forward(const Shape& s, const ar_rotation_t& r, bool inverse, const ar_heads_t& q,
            const ar_heads_t& k, const ar_heads_t& q_out, const ar_heads_t& k_out, bool norm,
            int weight_dtype, const void* q_weight, const void* k_weight, float eps, void* stream)
{
    const void* const weight[2] = {q_weight, k_weight};
    bool nothing = false;
    TRY(check_shape(s, &nothing));
    if (nothing)
        return AR_SUCCESS;
    Arrays all;
    HeadsArgs a{};
    TRY(add_heads(s, 0, q, false, 0, &all));
    TRY(add_heads(s, 1, k, false, 0, &all));
    TRY(add_heads(s, 0, q_out, true, 1, &all));
    TRY(add_heads(s, 1, k_out, true, 2, &all));
    TRY(add_turn(s, r, inverse, &all, &a.turn));
    if (norm)
        TRY(add_weights(s, weight_dtype, weight, &all));
    if (!disjoint(all))
        return AR_ERR_INVALID_USAGE;
    a.x[0] = array_of(q);
    a.x[1] = array_of(k);
    a.y[0] = array_of(q_out);
    a.y[1] = array_of(k_out);
    for (int side = 0; side < 2; ++side)
        a.weight[side] = s.heads[side] ? weight[side] : nullptr;
    a.heads0 = (uint32_t)s.heads[0];
    a.heads = fast_div((uint32_t)(s.heads[0] + s.heads[1]));
    a.tokens = fast_div((uint32_t)s.tokens);
    a.rows = (uint32_t)(s.batch * s.tokens * (s.heads[0] + s.heads[1]));
    a.dim = (uint32_t)s.dim;
    a.eps = eps;
    a.weight_f32 = weight_dtype == AR_FLOAT32;
    return done(launch_heads(s.dtype, norm, a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" int ar_rotary_frequencies(const ar_rotary_scheme_t* p, double* frequencies, double* factor)
{
    if (!p || !frequencies || !factor || p->rot_dim < 2 || p->rot_dim % 2 || p->rot_dim > kHeadMaxDim ||
        p->scaling < AR_SCALING_NONE || p->scaling > AR_SCALING_RAMP)
        return AR_ERR_INVALID_ARG;
    const auto finite_above = [](double v, double low) { return std::isfinite(v) && v > low; };
    const bool bands = p->scaling == AR_SCALING_BANDS, ramp = p->scaling == AR_SCALING_RAMP;
    if (!finite_above(p->base, 1.0) ||
        (p->scaling != AR_SCALING_NONE && !(std::isfinite(p->scale) && p->scale >= 1.0)) ||
        ((bands || ramp) && !finite_above(p->original, 0.0)) ||
        (bands && !(finite_above(p->low, 0.0) && finite_above(p->high, p->low))) ||
        (ramp && !(finite_above(p->slow, 0.0) && finite_above(p->fast, p->slow))) ||
        (p->scaling == AR_SCALING_BASE && p->rot_dim < 4))
        return AR_ERR_INVALID_ARG;
    const double pi = 3.14159265358979323846, r = (double)p->rot_dim;
    double base = p->base;
    if (p->scaling == AR_SCALING_BASE)
        base *= std::pow(p->scale, r / (r - 2.0));
    double lo = 0.0, hi = 0.0;
    if (ramp) {
        const auto at = [&](double turns) {
            return r * std::log(p->original / (2.0 * pi * turns)) / (2.0 * std::log(base));
        };
        lo = std::max(std::floor(at(p->fast)), 0.0);
        hi = std::min(std::ceil(at(p->slow)), r - 1.0);
    }
    for (size_t i = 0; i < p->rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * (double)i / r);
        double keep = 1.0;  // the share of the unscaled frequency
        if (p->scaling == AR_SCALING_LINEAR)
            keep = 0.0;
        else if (bands)
            keep = std::min(1.0, std::max(0.0, (p->original * f / (2.0 * pi) - p->low) / (p->high - p->low)));
        else if (ramp)
            keep = 1.0 - std::min(1.0, std::max(0.0, ((double)i - lo) / std::max(hi - lo, 0.001)));
        if (keep < 1.0)
            f *= keep + (1.0 - keep) / p->scale;
        frequencies[i] = f;
    }
    *factor = ramp ? 0.1 * std::log(p->scale) + 1.0 : 1.0;
    return AR_SUCCESS;
}

extern "C" int ar_rotary(const ar_rotary_t* p, void* stream)
{
    if (!p || p->rotation.rot_dim < 2)
        return AR_ERR_INVALID_ARG;
    const Shape s = {p->dtype, p->batch, p->tokens, {p->q_heads, p->k_heads}, p->dim};
    return forward(s, p->rotation, p->inverse != 0, p->q, p->k, p->q_out, p->k_out, false, p->dtype,
                   nullptr, nullptr, 0.0f, stream);
}

extern "C" int ar_head_rmsnorm(const ar_head_rmsnorm_t* p, void* stream)
{
    if (!p || bad_eps(p->eps))
        return AR_ERR_INVALID_ARG;
    const Shape s = {p->dtype, p->batch, p->tokens, {p->q_heads, p->k_heads}, p->dim};
    return forward(s, p->rotation, false, p->q, p->k, p->q_out, p->k_out, true, p->weight_dtype,
                   p->q_weight, p->k_weight, p->eps, stream);
}

extern "C" size_t ar_head_rmsnorm_backward_workspace(int ranks, size_t dim)
{
    if (ranks < 1 || ranks > kMaxRanks || dim < 1 || dim > kHeadMaxDim)
        return 0;
    return ((size_t)ranks * head_back_blocks(ranks) * 2 * dim * 4 + 255) / 256 * 256;
}

extern "C" int ar_head_rmsnorm_backward(const ar_head_rmsnorm_backward_t* p, void* stream)
{
    if (!p || bad_eps(p->eps) || p->ranks < 1 || p->ranks > kMaxRanks ||
        p->batch % (size_t)p->ranks)
        return AR_ERR_INVALID_ARG;
    const Shape s = {p->dtype, p->batch, p->tokens, {p->q_heads, p->k_heads}, p->dim};
    const void* const weight[2] = {p->q_weight, p->k_weight};
    float* const dweight[2] = {p->q_dweight, p->k_dweight};
    bool nothing = false;
    TRY(check_shape(s, &nothing));
    if (!s.heads[0] && !s.heads[1])
        return AR_SUCCESS;
    HeadsBackArgs a{};
    Arrays all;
    if (!nothing) {
        TRY(add_heads(s, 0, p->dq_out, false, 0, &all));
        TRY(add_heads(s, 1, p->dk_out, false, 0, &all));
        TRY(add_heads(s, 0, p->q, false, 0, &all));
        TRY(add_heads(s, 1, p->k, false, 0, &all));
        TRY(add_heads(s, 0, p->dq, true, 1 | 4, &all));
        TRY(add_heads(s, 1, p->dk, true, 2 | 8, &all));
        TRY(add_turn(s, p->rotation, true, &all, &a.turn));
        TRY(add_weights(s, p->weight_dtype, weight, &all));
        const size_t need = ar_head_rmsnorm_backward_workspace(p->ranks, p->dim);
        if (!p->workspace || p->workspace_bytes < need || (uintptr_t)p->workspace % 256)
            return AR_ERR_INVALID_ARG;
        all.own[all.nout] = 0;
        all.out[all.nout++] = block(p->workspace, need);
    }
    for (int side = 0; side < 2; ++side) {
        if (!s.heads[side])
            continue;
        if (!dweight[side] || misaligned(dweight[side], AR_FLOAT32))
            return AR_ERR_INVALID_ARG;
        all.own[all.nout] = 0;
        all.out[all.nout++] = block(dweight[side], (size_t)p->ranks * s.dim * 4);
        a.dweight[side] = dweight[side];
        a.weight[side] = weight[side];
        a.heads[side] = (uint32_t)s.heads[side];
        a.head[side] = fast_div((uint32_t)s.heads[side]);
    }
    if (!disjoint(all))
        return AR_ERR_INVALID_USAGE;
    a.dy[0] = array_of(p->dq_out);
    a.dy[1] = array_of(p->dk_out);
    a.x[0] = array_of(p->q);
    a.x[1] = array_of(p->k);
    a.dx[0] = array_of(p->dq);
    a.dx[1] = array_of(p->dk);
    a.partial = static_cast<float*>(p->workspace);
    a.tokens = fast_div(s.tokens ? (uint32_t)s.tokens : 1);
    a.rank_batches = (uint32_t)(s.batch / (size_t)p->ranks);
    a.rank_tokens = (uint32_t)(a.rank_batches * s.tokens);
    a.dim = (uint32_t)s.dim;
    a.ranks = p->ranks;
    a.eps = p->eps;
    a.weight_f32 = p->weight_dtype == AR_FLOAT32;
    return done(launch_heads_back(s.dtype, a, static_cast<hipStream_t>(stream)));
}
