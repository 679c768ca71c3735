// ar_ortho_host.cpp -- host side of the Newton-Schulz orthogonalisation: argument
// checks, the workspace's layout, and the sequence of products.
#include <algorithm>
#include <cmath>
#include <vector>

#include "ar_checks.h"
#include "ar_ortho.h"

using namespace ar;

namespace {

constexpr size_t kMaxSide = 65536;
constexpr int kMaxSteps = 64;

// Where a matrix's arrays lie in the workspace, in halves; X [m][n] with m <= n.
struct Layout {
    uint32_t m, n;
    uint64_t x[2], xt[2], a, b, each;  // each: one matrix's, all arrays
};

uint64_t whole(uint64_t halves) { return (halves + 127) / 128 * 128; }  // 256 bytes

Layout layout_of(size_t rows, size_t cols)
{
    Layout l;
    l.m = (uint32_t)std::min(rows, cols);
    l.n = (uint32_t)std::max(rows, cols);
    const uint64_t x = whole((uint64_t)l.m * 2 * padded(l.n)), xt = whole((uint64_t)l.n * 2 * padded(l.m)),
                   a = whole((uint64_t)l.m * 2 * padded(l.m));
    uint64_t at = whole(kNormParts * sizeof(double) / 2);  // the norm's parts come first
    for (uint64_t* p : {&l.x[0], &l.x[1]}) {
        *p = at;
        at += x;
    }
    for (uint64_t* p : {&l.xt[0], &l.xt[1]}) {
        *p = at;
        at += xt;
    }
    l.a = at;
    l.b = at + a;
    l.each = l.b + a;
    return l;
}

// Largest |p(s)| for s of [0, top], p = a s + b s^3 + c s^5 (odd), and largest
// |b s^2 + c s^4|: ends and the places where the slope is zero.
double largest(const float* k, double top, bool whole_step)
{
    const double a = k[0], b = k[1], c = k[2];
    const auto value = [&](double t) {  // t = s^2
        const double q = t * (b + t * c);
        return std::fabs(whole_step ? std::sqrt(t) * (a + q) : q);
    };
    double most = value(top * top);
    const auto at = [&](double t) {
        if (t > 0.0 && t < top * top)
            most = std::max(most, value(t));
    };
    if (whole_step) {  // a + 3 b t + 5 c t^2 = 0
        const double d = 9.0 * b * b - 20.0 * a * c;
        if (c != 0.0 && d >= 0.0) {
            at((-3.0 * b + std::sqrt(d)) / (10.0 * c));
            at((-3.0 * b - std::sqrt(d)) / (10.0 * c));
        } else if (b != 0.0) {
            at(-a / (3.0 * b));
        }
    } else if (c != 0.0) {  // b + 2 c t = 0
        at(-b / (2.0 * c));
    }
    return most;
}

// The exponent that leaves values up to `most` at 2^kOrthoTop.
int exponent(double most)
{
    return kOrthoTop - (most > 0.0 ? std::max(-100, std::ilogb(most) + 1) : -100);
}

// Bytes ahead of the matrices' arrays: the tickets and, where a side is long
// enough for products to go by parts, their slots.
size_t shared_bytes(const Layout& l)
{
    return kOrthoTickets * 4 +
           (padded(l.n) >= kOrthoPartPieces * 2 * kPiece ? kOrthoSlots * kOrthoSlotBytes : 0);
}

// Whether two matrices share a byte; rows of one stride may lie in turn.
bool meet(uintptr_t x, uintptr_t y, uint64_t rows, uint64_t len, uint64_t step_x, uint64_t step_y)
{
    if (x + (rows - 1) * step_x + len <= y || y + (rows - 1) * step_y + len <= x)
        return false;
    if (step_x != step_y || rows == 1)
        return true;
    const uint64_t d = y >= x ? (y - x) % step_x : (step_x - (x - y) % step_x) % step_x;
    return d < len || d + len > step_x;
}

}  // namespace

extern "C" size_t ar_orthogonalize_workspace(size_t count, size_t rows, size_t cols)
{
    if (rows > kMaxSide || cols > kMaxSide || !count || !rows || !cols)
        return 0;
    const Layout l = layout_of(rows, cols);
    return shared_bytes(l) + l.each * 2 * std::min<size_t>(count, kOrthoBatch);
}

extern "C" int ar_orthogonalize(const ar_orthogonalize_t* args, void* stream)
{
    if (!args)
        return AR_ERR_INVALID_ARG;
    ar_orthogonalize_t p = *args;
    if (!stream_type(p.dtype) || !(p.eps >= 0.0f) || std::isinf(p.eps) || !std::isfinite(p.scale) ||
        p.steps < 1 || p.steps > kMaxSteps || p.rows > kMaxSide || p.cols > kMaxSide ||
        p.count > ((size_t)1 << 24) || !p.coefficients)
        return AR_ERR_INVALID_ARG;
    for (int i = 0; i < 3 * p.steps; ++i)
        if (!std::isfinite(p.coefficients[i]))
            return AR_ERR_INVALID_ARG;
    if (!p.count || !p.rows || !p.cols)
        return AR_SUCCESS;
    if (p.rows == 1)
        p.x_stride = p.out_stride = p.cols;
    if (!p.x || !p.out || p.x_stride < p.cols || p.out_stride < p.cols ||
        p.x_stride > kMaxElems / p.rows || p.out_stride > kMaxElems / p.rows)
        return AR_ERR_INVALID_ARG;
    const Layout l = layout_of(p.rows, p.cols);
    const size_t shared = shared_bytes(l);
    if (!p.workspace || p.workspace_bytes < shared + l.each * 2 || (uintptr_t)p.workspace % 256)
        return AR_ERR_INVALID_ARG;
    const size_t room = std::min<size_t>(
        std::min<size_t>((p.workspace_bytes - shared) / (l.each * 2), p.count), kOrthoBatch);
    for (size_t i = 0; i < p.count; ++i)
        if (!p.x[i] || !p.out[i] || misaligned(p.x[i], p.dtype) || misaligned(p.out[i], p.dtype))
            return AR_ERR_INVALID_ARG;

    // how large X and b A + c A A get, step by step: their exponents
    std::vector<int> ex, eb, ea;
    try {
        ex.resize(p.steps + 1);
        ea.resize(p.steps);
        eb.resize(p.steps);
        const size_t z = size_of(p.dtype);
        const uint64_t len = p.cols * z, step_x = p.x_stride * z, step_out = p.out_stride * z;
        // out against everything, in order of address
        struct Item {
            uintptr_t at;
            size_t i;
            bool out;
        };
        std::vector<Item> items;
        items.reserve(2 * p.count);
        for (size_t i = 0; i < p.count; ++i) {
            items.push_back({(uintptr_t)p.x[i], i, false});
            items.push_back({(uintptr_t)p.out[i], i, true});
        }
        std::sort(items.begin(), items.end(), [](const Item& x, const Item& y) { return x.at < y.at; });
        const uint64_t reach_x = (p.rows - 1) * step_x + len, reach_out = (p.rows - 1) * step_out + len;
        const uintptr_t ws = (uintptr_t)p.workspace, ws_end = ws + shared + room * l.each * 2;
        for (size_t i = 0; i < items.size(); ++i) {
            const Item& v = items[i];
            const uint64_t reach = v.out ? reach_out : reach_x;
            if (v.at < ws_end && ws < v.at + reach)
                return AR_ERR_INVALID_USAGE;
            for (size_t j = i + 1; j < items.size() && items[j].at < v.at + reach; ++j) {
                const Item& w = items[j];
                if (!v.out && !w.out)
                    continue;
                const bool own = v.i == w.i && v.out != w.out && v.at == w.at && step_x == step_out;
                if (!own && meet(v.at, w.at, p.rows, len, v.out ? step_out : step_x,
                                 w.out ? step_out : step_x))
                    return AR_ERR_INVALID_USAGE;
            }
        }
    } catch (...) {
        return AR_ERR_INTERNAL;
    }
    double top = 1.0;  // of X's singular values
    for (int i = 0; i < p.steps; ++i) {
        ex[i] = exponent(top);
        ea[i] = exponent(top * top);
        eb[i] = exponent(largest(p.coefficients + 3 * i, top, false));
        top = largest(p.coefficients + 3 * i, top, true);
        if (!(top <= 65536.0))
            return AR_ERR_UNSUPPORTED;
    }
    ex[p.steps] = 0;

    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool tall = p.rows > p.cols;
    _Float16* const w = static_cast<_Float16*>(p.workspace) + shared / 2;
    uint32_t* const tickets = static_cast<uint32_t*>(p.workspace);
    for (size_t first = 0; first < p.count; first += room) {
        const int count = (int)std::min(room, p.count - first);
        OrthoPointers in{}, out{};
        for (int i = 0; i < count; ++i) {
            in.p[i] = p.x[first + i];
            out.p[i] = p.out[first + i];
        }
        OrthoSplitArgs split{};
        split.parts = reinterpret_cast<double*>(w);
        split.tickets = tickets;
        split.rowwise = w + (tall ? l.xt[0] : l.x[0]);
        split.colwise = w + (tall ? l.x[0] : l.xt[0]);
        split.each = l.each;
        split.stride = p.x_stride;
        split.rows = (uint32_t)p.rows;
        split.cols = (uint32_t)p.cols;
        split.bf16 = p.dtype == AR_BF16;
        split.eps = p.eps;
        split.up = std::ldexp(1.0, ex[0]);
        hipError_t e = launch_ortho_split(in, count, split, s);
        for (int i = 0; i < p.steps && e == hipSuccess; ++i) {
            const float* k = p.coefficients + 3 * i;
            const int now = i & 1;
            const bool last = i + 1 == p.steps;
            OrthoProductArgs g{};
            g.each = l.each;
            g.tickets = tickets;
            g.slots = reinterpret_cast<float*>(tickets + kOrthoTickets);
            g.bf16 = p.dtype == AR_BF16;
            // A = X X^T
            g.p = g.q = w + l.x[now];
            g.c = g.ct = w + l.a;
            g.m = g.n = l.m;
            g.k = padded(l.n) / kPiece;
            g.symmetric = 1;
            g.s_acc = (float)std::ldexp(1.0, ea[i] - 2 * ex[i]);
            e = launch_ortho_product(out, count, g, s);
            if (e != hipSuccess)
                break;
            // B = b A + c A A
            g.p = g.q = g.dt = w + l.a;
            g.c = g.ct = w + l.b;
            g.k = padded(l.m) / kPiece;
            g.s_acc = (float)std::ldexp((double)k[2], eb[i] - 2 * ea[i]);
            g.s_add = (float)std::ldexp((double)k[1], eb[i] - ea[i]);
            e = launch_ortho_product(out, count, g, s);
            if (e != hipSuccess)
                break;
            // X = a X + B X
            g.p = w + l.b;
            g.q = w + l.xt[now];
            g.dt = w + l.xt[now];
            g.c = w + l.x[!now];
            g.ct = w + l.xt[!now];
            g.n = l.n;
            g.symmetric = 0;
            const double up = std::ldexp(last ? (double)p.scale : 1.0, ex[i + 1] - ex[i]);
            g.s_acc = (float)std::ldexp(up, -eb[i]);
            g.s_add = (float)((double)k[0] * up);
            g.last = last;
            g.transposed = tall;
            g.out_stride = p.out_stride;
            e = launch_ortho_product(out, count, g, s);
        }
        if (e != hipSuccess)
            return done(e);
    }
    return AR_SUCCESS;
}
