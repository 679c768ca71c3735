// ar_ortho_host.cpp -- host side of the Newton-Schulz orthogonalisation: argument
// checks, the workspace's layout, and the sequence of products.
#include <algorithm>
#include <cmath>
#include <deque>
#include <map>
#include <utility>
#include <vector>

#include "ar_checks.h"
#include "ar_ortho.h"

using namespace ar;

namespace {

constexpr size_t kMaxSide = 65536;

// Where a matrix's arrays lie in the workspace, in halves; X [m][n] with m <= n.
struct Layout {
    uint32_t m, n;
    bool merged;
    uint64_t x[2], xt[2], square[5], each;  // each: one matrix's, all arrays
};

// Steps go by groups of up to three where the long side is this much the longer
// one, and the matrix large: a group multiplies X twice, by its transpose and by
// the product of the steps' polynomials, and does the rest on the short side's
// square matrices.  A group of g saves 4 (g - 1) m^2 n operations, and makes 6
// (g - 1) m^3 more, whose tiles fill the card better and write no transpose.  Five
// steps, by groups and one by one, float32: 4096 x 5734 4.74 and 5.30 ms, 4096 x 8192
// 5.39 and 6.42, 2048 x 4096 1127 and 1205 us, eight 1024 x 1433 1045 and 1102, but one
// alone 260 and 253, 512 x 1024 177 and 170, 160 x 320 114 and 111.  (4096 x 8192 bfloat16, whose
// groups may be larger: 4.91 ms.)  The number of matrices has no say, as the
// workspace's layout is by the matrix.
constexpr bool merges(uint32_t m, uint32_t n)
{
    return (uint64_t)n * 10 >= (uint64_t)m * 13 && (uint64_t)m * n >= 1u << 20;
}
constexpr int kMergeMost = 3;

uint64_t whole(uint64_t halves) { return (halves + 127) / 128 * 128; }  // 256 bytes

Layout layout_of(size_t rows, size_t cols)
{
    Layout l;
    l.m = (uint32_t)std::min(rows, cols);
    l.n = (uint32_t)std::max(rows, cols);
    const uint64_t x = whole((uint64_t)l.m * 2 * padded(l.n)), xt = whole((uint64_t)l.n * 2 * padded(l.m)),
                   a = whole((uint64_t)l.m * 2 * padded(l.m));
    uint64_t at = whole((kNormParts + 1) * sizeof(double) / 2);  // the norm's parts come first
    for (uint64_t* p : {&l.x[0], &l.x[1]}) {
        *p = at;
        at += x;
    }
    for (uint64_t* p : {&l.xt[0], &l.xt[1]}) {
        *p = at;
        at += xt;
    }
    l.merged = merges(l.m, l.n);
    for (int i = 0; i < (l.merged ? 5 : 2); ++i) {
        l.square[i] = at;
        at += a;
    }
    l.each = at;
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

// Largest |a + b s^2 + c s^4| for s of [0, top].
double steepest(const float* k, double top)
{
    const double a = k[0], b = k[1], c = k[2], t = top * top;
    double most = std::max(std::fabs(a), std::fabs(a + t * (b + t * c)));
    if (c != 0.0 && -b / (2.0 * c) > 0.0 && -b / (2.0 * c) < t)
        most = std::max(most, std::fabs(a - b * b / (4.0 * c)));
    return most;
}

// Largest |f(s)| for s of [0, top], of polynomials of low degree: by samples, that
// miss less than a hundredth of it (an exponent has room for three times).
template <class F>
double sampled(double top, F f)
{
    double most = 0.0;
    for (int i = 0; i <= 256; ++i)
        most = std::max(most, std::fabs(f(top * i / 256)));
    return most;
}

double q_of(const float* k, double s) { return k[0] + s * s * (k[1] + s * s * k[2]); }

// How much a step can widen an error of A = X X^T: the largest slope of s^2 -> p(s)^2.
double widening(const float* k, double top)
{
    return sampled(top, [&](double s) {
        return q_of(k, s) * (k[0] + s * s * (3.0 * k[1] + s * s * 5.0 * k[2]));
    });
}

// The power of two that values up to `most` stay below, and the exponent that
// leaves it at 2^kOrthoTop.
int power(double most)
{
    return most > 0.0 ? std::min(2000, std::max(-100, std::ilogb(most) + 1)) : -100;
}
int exponent(double most) { return kOrthoTop - power(most); }

// Bytes ahead of the matrices' arrays: the tickets and, where a side is long
// enough for products to go by parts, their slots.
size_t shared_bytes(const Layout& l)
{
    return kOrthoTickets * 4 +
           (padded(l.n) >= kOrthoPartPieces * 2 * kPiece ? kOrthoSlots * kOrthoSlotBytes : 0);
}

// Matrices of one kind (inputs or outputs) that reach past the address a walk over
// all of them has come to, by where their rows begin modulo the rows' distance.
// (Rows that lie in turn in one array: every matrix reaches past every other one,
// and is next to two of them there.)
class Reaching {
public:
    Reaching(uint64_t reach, uint64_t step) : reach_(reach), step_(step) {}
    void add(uintptr_t at, size_t i)
    {
        order_.push_back({at, by_.insert({at % step_, {at, i}})});
    }
    // leaves out what ends at `at` or ahead of it
    void walk_to(uintptr_t at)
    {
        for (; !order_.empty() && order_.front().first + reach_ <= at; order_.pop_front())
            by_.erase(order_.front().second);
    }
    // whether any but matrix `i` at this address shares a byte with rows of `len`
    // bytes, `step` apart; rows of another distance are taken to
    bool meets(uintptr_t at, uint64_t len, uint64_t step, size_t i) const
    {
        if (by_.empty())
            return false;
        if (step != step_)
            return true;
        const auto other = [&](uint64_t from, uint64_t to) {  // beginning in [from, to)
            for (auto v = by_.lower_bound(from); v != by_.end() && v->first < to; ++v)
                if (v->second.first != at || v->second.second != i)
                    return true;
            return false;
        };
        const uint64_t r = at % step, low = r + 1, high = r + len;  // r - len < beginning < r + len
        return other(low > len ? low - len : 0, std::min(high, step)) ||
               (low < len && other(step + low - len, step)) || (high > step && other(0, high - step));
    }

private:
    typedef std::multimap<uint64_t, std::pair<uintptr_t, size_t>> By;
    uint64_t reach_, step_;
    By by_;
    std::deque<std::pair<uintptr_t, By::iterator>> order_;
};

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
        p.steps < 1 || p.steps > kOrthoMaxSteps || p.rows > kMaxSide || p.cols > kMaxSide ||
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
    // (matrices that stay in LDS leave the workspace alone)
    const bool small = ortho_small(l.m, l.n);
    const size_t held = small ? kOrthoBatch : (p.workspace_bytes - shared) / (l.each * 2);
    const size_t room = std::min<size_t>(std::min<size_t>(held, p.count), kOrthoBatch);
    for (size_t i = 0; i < p.count; ++i)
        if (!p.x[i] || !p.out[i] || misaligned(p.x[i], p.dtype) || misaligned(p.out[i], p.dtype))
            return AR_ERR_INVALID_ARG;

    // how large X and b A + c A A get, step by step, and their exponents
    std::vector<int> ex, eb, ea, down, down_b;  // down, down_b: OrthoLift's now and b
    std::vector<double> tops;  // of X's singular values
    try {
        ex.resize(p.steps + 1);
        ea.resize(p.steps);
        eb.resize(p.steps);
        down.resize(p.steps + 1);
        down_b.resize(p.steps);
        tops.resize(p.steps + 1);
        const size_t z = size_of(p.dtype);
        const uint64_t len = p.cols * z, step_x = p.x_stride * z, step_out = p.out_stride * z;
        // out against everything, in order of address; out[i] may be x[i]
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
        const uintptr_t ws = (uintptr_t)p.workspace, ws_end = ws + shared + (small ? 1 : room) * l.each * 2;
        Reaching ins(reach_x, step_x), outs(reach_out, step_out);
        for (const Item& v : items) {
            if (v.at < ws_end && ws < v.at + (v.out ? reach_out : reach_x))
                return AR_ERR_INVALID_USAGE;
            ins.walk_to(v.at);
            outs.walk_to(v.at);
            const uint64_t step = v.out ? step_out : step_x;
            if (outs.meets(v.at, len, step, v.out ? SIZE_MAX : v.i) ||
                (v.out && ins.meets(v.at, len, step, v.i)))
                return AR_ERR_INVALID_USAGE;
            (v.out ? outs : ins).add(v.at, v.i);
        }
    } catch (...) {
        return AR_ERR_INTERNAL;
    }
    double top = tops[0] = 1.0, grown = 1.0;  // grown: at most, of an X that is small throughout
    for (int i = 0; i < p.steps; ++i) {
        const float* k = p.coefficients + 3 * i;
        const double b_top = largest(k, top, false);
        ex[i] = exponent(top);
        ea[i] = exponent(top * top);
        eb[i] = exponent(b_top);
        down[i] = std::max(0, power(grown) - power(top));
        // of b A + c A A, against A
        const double slope = std::max(std::fabs((double)k[1]), std::fabs(k[1] + top * top * k[2]));
        down_b[i] = std::max(0, 2 * power(top) + power(slope) - power(b_top));
        grown *= steepest(k, top);
        top = tops[i + 1] = largest(k, top, true);
        if (!(top <= 65536.0))
            return AR_ERR_UNSUPPORTED;
    }
    ex[p.steps] = 0;
    down[p.steps] = kOrthoGround;

    // a small result's power of two is its own, not the last product's factors'
    const double result = std::fabs((double)p.scale) * top;
    const int ends = power(result) < -32 ? power(result) : 0;
    const double own_scale = std::ldexp((double)p.scale, -ends);
    // what a step's sums and addends are multiplied by: coefficients, exponents, and
    // in the end the scale
    struct Factors {
        float a, b_acc, b_add, x_acc, x_add;
    };
    const auto factors = [&](int i) {
        const float* k = p.coefficients + 3 * i;
        const double up = std::ldexp(i + 1 == p.steps ? own_scale : 1.0, ex[i + 1] - ex[i]);
        return Factors{(float)std::ldexp(1.0, ea[i] - 2 * ex[i]),
                       (float)std::ldexp((double)k[2], eb[i] - 2 * ea[i]),
                       (float)std::ldexp((double)k[1], eb[i] - ea[i]), (float)std::ldexp(up, -eb[i]),
                       (float)((double)k[0] * up)};
    };
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
        if (small) {
            OrthoSmallArgs a{};
            a.x_stride = p.x_stride;
            a.out_stride = p.out_stride;
            a.rows = (uint32_t)p.rows;
            a.cols = (uint32_t)p.cols;
            a.bf16 = p.dtype == AR_BF16;
            a.steps = p.steps;
            a.eps = p.eps;
            a.ends = ends;
            a.up = std::ldexp(1.0, ex[0]);
            for (int i = 0; i < p.steps; ++i) {
                const Factors f = factors(i);
                a.step[i] = {f.a, f.b_acc, f.b_add, f.x_acc, f.x_add};
                a.lift[i] = (short)std::min(down[i], kOrthoSmallGround);
                a.lift_b[i] = (short)std::min(down_b[i], kOrthoSmallGround);
            }
            a.lift[p.steps] = kOrthoSmallGround;
            const hipError_t e = launch_ortho_small(in, out, count, a, s);
            if (e != hipSuccess)
                return done(e);
            continue;
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
        OrthoProductArgs g{};
        g.each = l.each;
        g.tickets = tickets;
        g.down = reinterpret_cast<const int*>(split.parts + kNormParts);
        g.slots = reinterpret_cast<float*>(tickets + kOrthoTickets);
        g.bf16 = p.dtype == AR_BF16;
        g.transposed = tall;
        g.out_stride = p.out_stride;
        // A symmetric product of square arrays: to = acc p q (+ add d + diag I)
        const auto square = [&](const _Float16* x, const _Float16* y, const _Float16* d, uint64_t to,
                                uint32_t pieces, double acc, double add, double diag,
                                const OrthoLift& lift) {
            if (e != hipSuccess)
                return;
            OrthoProductArgs c = g;
            c.p = x;
            c.q = y;
            c.dt = d;
            c.c = c.ct = w + to;
            c.m = c.n = l.m;
            c.k = pieces;
            c.symmetric = 1;
            c.s_acc = (float)acc;
            c.s_add = (float)add;
            c.diag = (float)diag;
            c.lift = lift;
            e = launch_ortho_product(out, count, c, s);
        };
        const uint32_t long_k = padded(l.n) / kPiece, short_k = padded(l.m) / kPiece;
        const uint64_t A = l.square[0];
        int now = 0;
        for (int i = 0; i < p.steps; now = !now) {
            const float* k = p.coefficients + 3 * i;
            int group = 1;
            for (double wide = 1.0; l.merged && group < kMergeMost && i + group < p.steps; ++group) {
                // what the group's later steps take for A is off by that much more: 2^-23
                // widened by 256 is a part in 128 of bfloat16's own rounding (4096 x 8192: 4.88
                // ms, by 16 5.33, 1.660e-3 off the 64-bit result either way)
                wide *= widening(k + 3 * (group - 1), tops[i + group - 1]);
                if (!(wide <= (p.dtype == AR_BF16 ? 256.0 : 16.0)))
                    break;
            }
            const int end = i + group;
            const bool last = end == p.steps;
            const double scale = last ? own_scale : 1.0;
            const _Float16 *x = w + l.x[now], *xt = w + l.xt[now];
            square(x, x, nullptr, A, long_k, std::ldexp(1.0, ea[i] - 2 * ex[i]), 0.0, 0.0, {});
            // the last product's factor of X: B, beside a X, or the group's polynomial F
            uint64_t factor = l.square[1];
            int factor_e = eb[i];
            if (group == 1) {
                const Factors f = factors(i);
                square(w + A, w + A, w + A, factor, short_k, f.b_acc, f.b_add, 0.0,
                       {down[i], 0, down_b[i], {-4, 0, 1}, {-2, 0, 1}});
            } else {
                uint64_t T = l.square[2], Q = factor, other = l.square[3], spare = l.square[4];
                double f_top = 1.0;
                for (int j = i;; ++j) {
                    const float* kj = p.coefficients + 3 * j;
                    // Q = a I + b A + c A A
                    const int eq = exponent(sampled(tops[j], [&](double v) { return q_of(kj, v); }));
                    square(w + A, w + A, w + A, Q, short_k, std::ldexp((double)kj[2], eq - 2 * ea[j]),
                           std::ldexp((double)kj[1], eq - ea[j]), std::ldexp((double)kj[0], eq),
                           {down[j], 0, 0, {-4, 0, 0}, {-2, 0, 0}});
                    f_top *= sampled(tops[j], [&](double v) { return q_of(kj, v); });
                    const int ef = exponent(f_top);
                    if (j == i) {
                        factor_e = eq;  // F = Q
                    } else {            // F = Q F
                        const uint64_t to = j == i + 1 ? spare : T;
                        square(w + Q, w + factor, nullptr, to, short_k, std::ldexp(1.0, ef - eq - factor_e),
                               0.0, 0.0, {});
                        factor = to;
                        factor_e = ef;
                    }
                    if (j + 1 == end)
                        break;
                    // A of the next step is Q A Q, by T = Q A: they commute
                    const int et = exponent(tops[j] * tops[j + 1]);
                    const OrthoLift lift = {down[j], down[j + 1], 0, {-1, 1, 0}, {}};
                    square(w + Q, w + A, nullptr, T, short_k, std::ldexp(1.0, et - eq - ea[j]), 0.0, 0.0,
                           lift);
                    square(w + Q, w + T, nullptr, A, short_k, std::ldexp(1.0, ea[j + 1] - eq - et), 0.0,
                           0.0, lift);
                    std::swap(Q, other);
                }
            }
            if (e != hipSuccess)
                break;
            OrthoProductArgs c = g;
            c.p = w + factor;
            c.q = xt;
            c.c = w + l.x[!now];
            c.ct = w + l.xt[!now];
            c.m = l.m;
            c.n = l.n;
            c.k = short_k;
            c.last = last;
            c.ends = last ? ends : 0;
            if (group == 1) {  // X = a X + B X
                const Factors f = factors(i);
                c.dt = xt;
                c.s_acc = f.x_acc;
                c.s_add = f.x_add;
                c.lift = {down[i], down[end], down_b[i], {-1, 1, -1}, {-1, 1, 0}};
            } else {  // X = F X
                c.s_acc = (float)std::ldexp(scale, ex[end] - ex[i] - factor_e);
                c.lift = {down[i], down[end], 0, {-1, 1, 0}, {}};
            }
            e = launch_ortho_product(out, count, c, s);
            i = end;
        }
        if (e != hipSuccess)
            return done(e);
    }
    return AR_SUCCESS;
}
