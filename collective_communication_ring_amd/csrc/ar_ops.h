// ar_ops.h -- definitions shared by the host side and the HIP kernels of the
// operators around the collectives: RMS norm (ar_norm.hip), its backward pass
// (ar_norm_back.hip), gradient norm and clipping (ar_grad.hip).  Not part of
// the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ar.h"

namespace ar {

// One forward norm.  h(t, c) = the sum of `parts` rows + the residual's row.
// parts == 1: x(t, c) at x[t * x_stride + c].  Else the parts are the rank
// rows of a reduce-scatter's send: rank p's value of token t at
// x[p * part_stride + t * cols + c], folded in the ring's order -- from the
// successor of the token's owner (t / tokens_per_rank) round to the owner.
struct NormArgs {
    const void* x;
    const void* residual;  // or NULL
    const void* weight;
    void* sum;             // or NULL
    void* y;
    float* scale;          // e4m3 only: [rows][groups]
    float* rstd;           // or NULL
    uint64_t rows;
    uint64_t x_stride;
    uint64_t res_stride;
    uint64_t sum_stride;
    uint64_t y_stride;
    uint64_t part_stride;
    uint64_t tokens_per_rank;
    uint32_t cols;
    uint32_t group;        // e4m3: columns per scale (cols: one for the row)
    uint32_t groups;       // scales per row
    int parts;
    float divisor;         // 1, or the number of ranks (average)
    float eps;
    int weight_f32;        // weight is float32 (else of the stream's type)
};

struct NormBackArgs {
    const void* dy;
    const void* x;
    const void* weight;
    const void* dsum;      // or NULL
    const float* rstd;
    void* dx;
    float* dweight;        // [ranks][cols]
    float* partial;        // [ranks][blocks][cols]
    uint64_t rows_per_rank;
    uint64_t dy_stride;
    uint64_t x_stride;
    uint64_t dsum_stride;
    uint64_t dx_stride;
    uint32_t cols;
    int ranks;
    int blocks;            // partial rows of dweight per rank
    int weight_f32;
};

constexpr uint64_t kNormMaxCols = 1u << 30;  // 32-bit column indexes in the kernels
constexpr int kNormBackMaxBlocks = 512;      // partial rows of dweight per rank, at most

// Partial rows of dweight for one rank's rows (the same for every type, so
// that the workspace is known from sizes alone).
int norm_back_blocks(uint64_t rows_per_rank, int ranks);

hipError_t launch_rmsnorm(int dtype, bool e4m3, const NormArgs& a, hipStream_t s);
hipError_t launch_rmsnorm_back(int dtype, const NormBackArgs& a, hipStream_t s);

// ---- gradient lists ---------------------------------------------------------

// A table of spans passed by value in a launch's kernel arguments (no copy to
// the device, and a captured graph keeps its own): 4 KiB of arguments hold
// this many.
constexpr int kSpansPerLaunch = 128;

// A span is cut into tiles of kGradTileVecs 16-byte vectors, counted from its
// first 16-byte boundary; the elements before that boundary and after the last
// whole vector belong to its first tile.  Every span has a tile.
constexpr uint32_t kGradTileVecs = 1024;

struct SpanTable {
    const void* src[kSpansPerLaunch];
    uint64_t count[kSpansPerLaunch];
    uint32_t first[kSpansPerLaunch];  // first tile of the span; bit 31: bfloat16
    uint32_t tiles;                   // of all spans of this table
    int n;
};

struct SpanPairTable {
    const void* src[kSpansPerLaunch];
    void* dst[kSpansPerLaunch];
    uint64_t count[kSpansPerLaunch];
    uint32_t first[kSpansPerLaunch];
    uint32_t tiles;
    int n;
};

constexpr int kGradMaxBlocks = 2048;  // slots of partial sums in a communicator's workspace

// Sums of squares of one table's spans.  Slots [0, live) of `partial` hold the
// sums of the tables before it, to which this one adds.  `norm` (the last
// table): the root of the sum of all slots goes there.
hipError_t launch_grad_norm(const SpanTable& t, double* partial, int live, int grid,
                            uint32_t* ticket, float* norm, hipStream_t s);
hipError_t launch_grad_clip(const SpanPairTable& t, const float* norm, float max_norm, int grid,
                            hipStream_t s);

// Tables of a list, one after the other (ar_ops.cpp).  ar_grad_norm's work.
int grad_norm_run(const ar_span_t* grads, size_t n, float* norm, double* partial, uint32_t* ticket,
                  hipStream_t s, hipError_t* err);
// Argument checks of a norm, and its kernel arguments.  parts > 1: p.x is the
// reduce-scatter's send of that many rank rows of p.rows tokens each.
int norm_prepare(ar_rmsnorm_t p, int parts, NormArgs* out, bool* noop);

}  // namespace ar
