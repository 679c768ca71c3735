// ar_ops.cpp -- host side of the operators around the collectives: argument
// checks, workspace sizes, and the tables of gradient lists.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <iterator>
#include <vector>

#include "ar_checks.h"
#include "ar_internal.h"
#include "ar_ops.h"

using namespace ar;

namespace {

// An array of `rows` rows of `len` bytes, `stride` bytes apart.
struct Rows {
    uintptr_t at;
    uint64_t rows, len, stride;
};

Rows rows_of(const void* p, size_t rows, size_t cols, size_t stride, int dtype)
{
    const size_t z = size_of(dtype);
    return {(uintptr_t)p, rows, cols * z, stride * z};
}

// Whether two arrays share a byte (a NULL one shares none).  Rows of one
// stride may lie between each other's; with two strides the extents decide.
bool share(const Rows& a, const Rows& b)
{
    if (!a.at || !b.at || !a.rows || !b.rows)
        return false;
    if (a.at + (a.rows - 1) * a.stride + a.len <= b.at || b.at + (b.rows - 1) * b.stride + b.len <= a.at)
        return false;
    const uint64_t stride = a.rows > 1 ? a.stride : b.stride;
    if ((a.rows == 1 && b.rows == 1) || (a.rows > 1 && b.rows > 1 && a.stride != b.stride))
        return true;
    const uint64_t d = b.at >= a.at ? (b.at - a.at) % stride
                                    : (stride - (a.at - b.at) % stride) % stride;
    return d < a.len || d + b.len > stride;
}

// The same rows in the same type: an output may replace this input.
bool same(const Rows& a, const Rows& b)
{
    return a.at == b.at && a.len == b.len && (a.rows == 1 || a.stride == b.stride);
}

// Outputs against each other and against the inputs.  out[0 .. replacing) may
// have the array of one of in[0 .. replaced); the others are of another kind,
// whatever their address and length.
bool disjoint(const Rows* out, int nout, int replacing, const Rows* in, int nin, int replaced)
{
    for (int i = 0; i < nout; ++i) {
        for (int j = i + 1; j < nout; ++j)
            if (share(out[i], out[j]))
                return false;
        for (int j = 0; j < nin; ++j)
            if (share(out[i], in[j]) && !(i < replacing && j < replaced && same(out[i], in[j])))
                return false;
    }
    return true;
}

// Rows of `cols` elements `*stride` apart: the stride of a single row means
// nothing, else rows must not overlap and the array stay below kMaxElems.
bool bad_stride(size_t rows, size_t cols, size_t* stride)
{
    if (rows == 1)
        *stride = cols;
    return *stride < cols || *stride > kMaxElems / rows;
}

}  // namespace

namespace ar {

int norm_prepare(ar_rmsnorm_t p, int parts, NormArgs* out, bool* noop)
{
    *noop = false;
    if (!stream_type(p.dtype) || (p.out_dtype != p.dtype && p.out_dtype != AR_E4M3) ||
        (p.weight_dtype != p.dtype && p.weight_dtype != AR_FLOAT32))
        return AR_ERR_INVALID_ARG;
    if (!(p.eps >= 0.0f) || std::isinf(p.eps) || p.cols > kNormMaxCols || p.rows > kMaxElems)
        return AR_ERR_INVALID_ARG;
    const bool e4m3 = p.out_dtype == AR_E4M3;
    if (e4m3 && p.group != 0 && p.group != 32 && p.group != 64 && p.group != 128 && p.group != 256)
        return AR_ERR_INVALID_ARG;
    if (p.rows == 0 || p.cols == 0) {
        *noop = true;
        return AR_SUCCESS;
    }
    if (!p.x || !p.weight || !p.y || (e4m3 && !p.scale))
        return AR_ERR_INVALID_ARG;
    if (bad_stride(p.rows, p.cols, &p.x_stride) || bad_stride(p.rows, p.cols, &p.y_stride) ||
        (p.residual && bad_stride(p.rows, p.cols, &p.residual_stride)) ||
        (p.sum && bad_stride(p.rows, p.cols, &p.sum_stride)))
        return AR_ERR_INVALID_ARG;
    if (misaligned(p.x, p.dtype) || misaligned(p.residual, p.dtype) || misaligned(p.sum, p.dtype) ||
        misaligned(p.y, p.out_dtype) || misaligned(p.weight, p.weight_dtype) ||
        misaligned(p.scale, AR_FLOAT32) || misaligned(p.rstd, AR_FLOAT32))
        return AR_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = p.x;
    a.residual = p.residual;
    a.weight = p.weight;
    a.sum = p.sum;
    a.y = p.y;
    a.scale = e4m3 ? p.scale : nullptr;
    a.rstd = p.rstd;
    a.rows = p.rows;
    a.x_stride = p.x_stride;
    a.res_stride = p.residual_stride;
    a.sum_stride = p.sum_stride;
    a.y_stride = p.y_stride;
    a.cols = (uint32_t)p.cols;
    a.group = e4m3 && p.group && p.group < p.cols ? (uint32_t)p.group : (uint32_t)p.cols;
    a.groups = (a.cols + a.group - 1) / a.group;
    a.parts = parts;
    a.divisor = 1.0f;
    a.eps = p.eps;
    a.weight_f32 = p.weight_dtype == AR_FLOAT32;
    if (parts > 1) {
        a.part_stride = p.rows * p.cols;
        a.tokens_per_rank = p.rows / (size_t)parts;
    }
    const Rows res = rows_of(p.residual, p.rows, p.cols, p.residual_stride, p.dtype);
    const Rows x = parts > 1 ? rows_of(p.x, 1, (size_t)parts * p.rows * p.cols, 0, p.dtype)
                             : rows_of(p.x, p.rows, p.cols, p.x_stride, p.dtype);
    const Rows w = rows_of(p.weight, 1, p.cols, 0, p.weight_dtype);
    const Rows outs[] = {rows_of(p.y, p.rows, p.cols, p.y_stride, p.out_dtype),
                         rows_of(p.sum, p.rows, p.cols, p.sum_stride, p.dtype),
                         rows_of(a.scale, 1, p.rows * a.groups, 0, AR_FLOAT32),
                         rows_of(p.rstd, 1, p.rows, 0, AR_FLOAT32)};
    const Rows ins[] = {res, x, w};
    if (!disjoint(outs, 4, 2, ins, 3, parts > 1 ? 1 : 2))
        return AR_ERR_INVALID_USAGE;
    *out = a;
    return AR_SUCCESS;
}

}  // namespace ar

extern "C" int ar_rmsnorm(const ar_rmsnorm_t* args, void* stream)
{
    if (!args)
        return AR_ERR_INVALID_ARG;
    NormArgs a{};
    bool noop = false;
    const int rc = norm_prepare(*args, 1, &a, &noop);
    if (rc || noop)
        return rc;
    return done(launch_rmsnorm(args->dtype, args->out_dtype == AR_E4M3, a,
                               static_cast<hipStream_t>(stream)));
}

extern "C" size_t ar_rmsnorm_backward_workspace(int ranks, size_t rows, size_t cols)
{
    if (ranks < 1 || ranks > kMaxRanks || rows % (size_t)ranks || cols > kNormMaxCols)
        return 0;
    const size_t n = (size_t)ranks * norm_back_blocks(rows / (size_t)ranks, ranks) * cols * 4;
    return (n + 255) / 256 * 256;
}

extern "C" int ar_rmsnorm_backward(const ar_rmsnorm_backward_t* args, void* stream)
{
    if (!args)
        return AR_ERR_INVALID_ARG;
    ar_rmsnorm_backward_t p = *args;
    if (!stream_type(p.dtype) || (p.weight_dtype != p.dtype && p.weight_dtype != AR_FLOAT32) ||
        p.ranks < 1 || p.ranks > kMaxRanks || p.rows % (size_t)p.ranks || p.cols > kNormMaxCols ||
        p.rows > kMaxElems)
        return AR_ERR_INVALID_ARG;
    if (p.cols == 0)
        return AR_SUCCESS;
    if (!p.dweight || misaligned(p.dweight, AR_FLOAT32))
        return AR_ERR_INVALID_ARG;
    if (p.rows) {
        if (!p.dy || !p.x || !p.weight || !p.rstd || !p.dx || !p.workspace ||
            p.workspace_bytes < ar_rmsnorm_backward_workspace(p.ranks, p.rows, p.cols) ||
            (uintptr_t)p.workspace % 256)
            return AR_ERR_INVALID_ARG;
        if (bad_stride(p.rows, p.cols, &p.dy_stride) || bad_stride(p.rows, p.cols, &p.x_stride) ||
            bad_stride(p.rows, p.cols, &p.dx_stride) ||
            (p.dsum && bad_stride(p.rows, p.cols, &p.dsum_stride)))
            return AR_ERR_INVALID_ARG;
        if (misaligned(p.dy, p.dtype) || misaligned(p.x, p.dtype) || misaligned(p.dsum, p.dtype) ||
            misaligned(p.dx, p.dtype) || misaligned(p.weight, p.weight_dtype) ||
            misaligned(p.rstd, AR_FLOAT32))
            return AR_ERR_INVALID_ARG;
        const Rows outs[] = {
            rows_of(p.dx, p.rows, p.cols, p.dx_stride, p.dtype),
            rows_of(p.dweight, 1, (size_t)p.ranks * p.cols, 0, AR_FLOAT32),
            {(uintptr_t)p.workspace, 1, ar_rmsnorm_backward_workspace(p.ranks, p.rows, p.cols), 0}};
        const Rows ins[] = {rows_of(p.dy, p.rows, p.cols, p.dy_stride, p.dtype),
                            rows_of(p.x, p.rows, p.cols, p.x_stride, p.dtype),
                            rows_of(p.dsum, p.rows, p.cols, p.dsum_stride, p.dtype),
                            rows_of(p.weight, 1, p.cols, 0, p.weight_dtype),
                            rows_of(p.rstd, 1, p.rows, 0, AR_FLOAT32)};
        if (!disjoint(outs, 3, 1, ins, 5, 3))
            return AR_ERR_INVALID_USAGE;
    }
    NormBackArgs a{};
    a.dy = p.dy;
    a.x = p.x;
    a.weight = p.weight;
    a.dsum = p.dsum;
    a.rstd = p.rstd;
    a.dx = p.dx;
    a.dweight = p.dweight;
    a.partial = static_cast<float*>(p.workspace);
    a.rows_per_rank = p.rows / (size_t)p.ranks;
    a.dy_stride = p.dy_stride;
    a.x_stride = p.x_stride;
    a.dsum_stride = p.dsum_stride;
    a.dx_stride = p.dx_stride;
    a.cols = (uint32_t)p.cols;
    a.ranks = p.ranks;
    a.blocks = norm_back_blocks(a.rows_per_rank, p.ranks);
    a.weight_f32 = p.weight_dtype == AR_FLOAT32;
    return done(launch_rmsnorm_back(p.dtype, a, static_cast<hipStream_t>(stream)));
}

// ---- gradient lists ---------------------------------------------------------

namespace {

constexpr size_t kMaxSpan = (size_t)1 << 36;      // elements of a tensor: 256 GiB of float32
constexpr uint64_t kMaxTiles = 0xfffffffeu;       // of a table (2^24 of the largest tensor)

bool bad_span(const ar_span_t& s)
{
    return !stream_type(s.dtype) || s.count > kMaxSpan || ((uintptr_t)s.data & ~kSpanAddress) ||
           (s.count && (!s.data || misaligned(s.data, s.dtype)));
}

// The next table of a list from span *i on, empty spans left out.
// place(i, k, &shift): span i's output is that of entry k; false: not in this
// table.
template <class Table, class Place>
void next_table(const ar_span_t* in, size_t n, size_t* i, Table* t, Place place)
{
    t->tiles = 0;
    t->n = 0;
    for (; *i < n && t->n < Table::kSpans; ++*i) {
        const ar_span_t& s = in[*i];
        if (!s.count)
            continue;
        const uint64_t halves = s.count * size_of(s.dtype) / 2;
        const uint64_t tiles = (halves + kGradTileHalves - 1) / kGradTileHalves;
        uint32_t shift = 0;
        if (t->tiles + tiles > kMaxTiles || !place(*i, t->n, &shift))
            break;
        t->span[t->n] = pack_span(s.data, (uint32_t)(halves - (tiles - 1) * kGradTileHalves),
                                  s.dtype == AR_BF16, shift);
        t->first[t->n] = t->tiles;
        t->tiles += (uint32_t)tiles;
        ++t->n;
    }
    while (*i < n && !in[*i].count)
        ++*i;
    std::fill(t->first + t->n, std::end(t->first), 0xffffffffu);
}

// Workgroups for a table: a tile each while they are few.
int grid_for(uint32_t tiles)
{
    return (int)std::max<uint32_t>(1, std::min<uint32_t>(tiles, kGradMaxBlocks));
}

// A stretch of addresses.
struct Reach {
    uintptr_t lo, hi;
};

bool before(const Reach& x, const Reach& y) { return x.lo < y.lo; }

void sort_reaches(std::vector<Reach>* v)
{
    // tensors cut from one buffer come in order
    if (!std::is_sorted(v->begin(), v->end(), before))
        std::sort(v->begin(), v->end(), before);
}

// Whether an output shares bytes with another output, or with an input that is
// not its own in place.
bool clip_overlaps(const ar_span_t* in, const ar_span_t* out, size_t n, const float* norm)
{
    std::vector<Reach> reads, writes;
    reads.reserve(n);
    writes.reserve(n);
    for (size_t i = 0; i < n; ++i) {
        const size_t bytes = in[i].count * size_of(in[i].dtype);
        if (!bytes)
            continue;
        const uintptr_t a = (uintptr_t)in[i].data, b = (uintptr_t)out[i].data;
        if (a != b)
            reads.push_back({a, a + bytes});
        writes.push_back({b, b + bytes});
        if ((uintptr_t)norm < b + bytes && b < (uintptr_t)norm + sizeof(float))
            return true;
    }
    sort_reaches(&reads);
    sort_reaches(&writes);
    for (size_t k = 1; k < writes.size(); ++k)
        if (writes[k].lo < writes[k - 1].hi)
            return true;
    // the writes are disjoint now, so their ends are in order too: for a read,
    // the first that ends behind its start is the only one to look at
    auto w = writes.begin();
    for (const Reach& r : reads) {
        while (w != writes.end() && w->hi <= r.lo)
            ++w;
        if (w != writes.end() && w->lo < r.hi)
            return true;
    }
    return false;
}

}  // namespace

namespace ar {

int grad_norm_run(const ar_span_t* grads, size_t n, float* norm, void* scratch, hipStream_t s,
                  hipError_t* err)
{
    *err = hipSuccess;
    if (!norm || misaligned(norm, AR_FLOAT32) || (n && !grads))
        return AR_ERR_INVALID_ARG;
    for (size_t i = 0; i < n; ++i) {
        if (bad_span(grads[i]))
            return AR_ERR_INVALID_ARG;
        const uintptr_t at = (uintptr_t)grads[i].data, to = (uintptr_t)norm;
        if (to < at + grads[i].count * size_of(grads[i].dtype) && at < to + sizeof(float) &&
            grads[i].count)
            return AR_ERR_INVALID_USAGE;
    }
    int live = 0;
    size_t i = 0;
    do {  // a list of nothing has one table, of no spans: its norm is 0
        SpanTable<kNormSpans> t;
        next_table(grads, n, &i, &t, [](size_t, int, uint32_t*) { return true; });
        const int grid = grid_for(t.tiles);
        *err = launch_grad_norm(t, scratch, live, grid, i == n ? norm : nullptr, s);
        if (*err != hipSuccess)
            return AR_ERR_HIP;
        live = std::max(live, grid);
    } while (i < n);
    return AR_SUCCESS;
}

}  // namespace ar

extern "C" int ar_grad_clip(const ar_span_t* grads, const ar_span_t* out, size_t n,
                            const float* norm, float max_norm, void* stream)
{
    if (!(max_norm >= 0.0f) || !norm || misaligned(norm, AR_FLOAT32) || (n && (!grads || !out)))
        return AR_ERR_INVALID_ARG;
    for (size_t i = 0; i < n; ++i)
        if (bad_span(grads[i]) || bad_span(out[i]) || grads[i].count != out[i].count ||
            grads[i].dtype != out[i].dtype)
            return AR_ERR_INVALID_ARG;
    try {
        if (clip_overlaps(grads, out, n, norm))
            return AR_ERR_INVALID_USAGE;
    } catch (...) {
        return AR_ERR_INTERNAL;
    }
    hipStream_t st = static_cast<hipStream_t>(stream);
    for (size_t i = 0; i < n;) {
        // by distances, if the table so made holds more than one of addresses would
        size_t next = i;
        SpanTable<kNormSpans> t;
        SpanShifts by = {};
        int shifts = 0;
        next_table(grads, n, &next, &t, [&](size_t k, int, uint32_t* shift) {
            const uint64_t d = (uint64_t)(uintptr_t)out[k].data - (uint64_t)(uintptr_t)grads[k].data;
            while (*shift < (uint32_t)shifts && by.by[*shift] != d)
                ++*shift;
            if (*shift == kClipShifts)
                return false;
            if (*shift == (uint32_t)shifts)
                by.by[shifts++] = d;
            return true;
        });
        hipError_t e = hipSuccess;
        if (next == n || t.n >= kClipSpans) {
            if (t.n)
                e = launch_grad_clip(t, by, norm, max_norm, grid_for(t.tiles), st);
            i = next;
        } else {
            SpanTable<kClipSpans> u;
            SpanOutputs o;
            next_table(grads, n, &i, &u, [&](size_t k, int at, uint32_t*) {
                o.dst[at] = (uint64_t)(uintptr_t)out[k].data;
                return true;
            });
            e = launch_grad_clip(u, o, norm, max_norm, grid_for(u.tiles), st);
        }
        if (e != hipSuccess)
            return done(e);
    }
    return AR_SUCCESS;
}
