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
    uint64_t row0;         // this launch's first row (set by the launch)
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
    uint32_t lanes;        // threads per row (set by the launch)
    int exact;             // lanes hold a row without a rest (set by the launch)
    int stream;            // outputs larger than the L2s (set by the launch)
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
    uint32_t lanes;        // threads per row, and rows side by side in a workgroup
    uint32_t rows;         //   (set by the launch)
    int exact;             // lanes hold a row without a rest (set by the launch)
    int stream;            // dx is larger than the L2s (set by the launch)
};

constexpr int kMaxWaves = 16;                // waves that share a row, at most
constexpr uint64_t kNormMaxCols = 1u << 28;  // 32-bit column and thread numbers in a launch
// Threads of a launch of the forward norm, at most (a grid holds fewer than
// 2^32): more rows go by several launches.
constexpr uint64_t kNormMaxThreads = (uint64_t)1 << 31;
// Bytes of an output above which whole rows of it are stored non-temporally:
// what the 8 L2s hold.  bf16 8192 x 8192 with e4m3 output 82 -> 75 us, bf16 4097
// x 16384 107 -> 95 us; smaller outputs are left for whoever reads them next,
// and rows that do not fill their last lines lose by it (2568: 33 -> 35 us).
constexpr uint64_t kStreamBytes = (uint64_t)32 << 20;
// Partial rows of dweight of all ranks, at most: a workgroup of 16 waves on each
// CU, all resident (bf16 8192 x 8192: 92 us; 128 workgroups 137, 512 96; 8192 x
// 4096: 50, 70, 53; 8 ranks' 625 x 2049: 23, 32, 26).
constexpr int kNormBackMaxBlocks = 256;

// Partial rows of dweight for one rank's rows (the same for every type, so
// that the workspace is known from sizes alone).
int norm_back_blocks(uint64_t rows_per_rank, int ranks);

hipError_t launch_rmsnorm(int dtype, bool e4m3, NormArgs a, hipStream_t s);
hipError_t launch_rmsnorm_back(int dtype, NormBackArgs a, hipStream_t s);

// ---- gradient lists ---------------------------------------------------------

// A span is cut into tiles of kGradTileVecs 16-byte vectors from its first
// element on (at any alignment); the last tile may be cut short.
constexpr uint32_t kGradTileVecs = 1024;
constexpr uint32_t kGradTileHalves = kGradTileVecs * 8;  // in 16-bit units, as lengths are kept

// A table of spans is passed by value in a launch's kernel arguments: no copy
// to the device, and a captured graph keeps its own.  A span is packed into one
// word -- its address (48 bits), the 16-bit units of its last tile less one (13
// bits), which of kClipShifts distances its output lies at (2 bits), and
// whether it is bfloat16 -- so that 4 KiB of arguments hold kNormSpans of them,
// or kClipSpans with an output address each.  Outputs in place or cut from a
// few buffers as their inputs are need the distances alone: 291 tensors are
// clipped by one launch instead of two.
constexpr int kNormSpans = 312;
constexpr int kClipSpans = 184;
constexpr int kClipShifts = 4;
constexpr uint64_t kSpanAddress = ((uint64_t)1 << 48) - 1;
constexpr uint64_t kSpanBf16 = (uint64_t)1 << 63;
inline uint64_t pack_span(const void* p, uint32_t last_halves, bool bf16, uint32_t shift)
{
    return (uint64_t)(uintptr_t)p | (uint64_t)(last_halves - 1) << 48 | (uint64_t)shift << 61 |
           (bf16 ? kSpanBf16 : 0);
}

template <int N>
struct SpanTable {
    static constexpr int kSpans = N;
    uint64_t span[N];
    uint32_t first[(N + 63) / 64 * 64];  // first tile of the span; 2^32 - 1 past the last (whole
                                         // rounds of a wave's lanes)
    uint32_t tiles;                      // of all spans of this table
    int n;
};

// Where a table's outputs are: an address each, or the distances (modulo 2^64)
// from input to output.
struct SpanOutputs {
    uint64_t dst[kClipSpans];
};
struct SpanShifts {
    uint64_t by[kClipShifts];
};

// Workgroups of a launch, at most: 2 on each of 256 CUs.  They take the tiles
// in turn (tile t goes to workgroup t mod grid), so that the whole grid reads
// one stretch of memory at a time: 40 x 25 MiB of bfloat16 normed and clipped
// in 504 us (6.2 TB/s over its three passes), against 569 us with a stretch of
// its own for each workgroup.  1024 workgroups: the same there, and 15.1 us
// for a norm of 64 MiB against 14.3.
constexpr int kGradMaxBlocks = 512;
// Workgroups take tickets in groups of this many, each group's counter in a
// 128-byte line of its own, and the last of a group takes one for the group:
// an atomic on one address from every workgroup costs ~10 ns each (a 64 MiB
// norm by 2048 workgroups: 34 us, 16 us with the groups).
constexpr int kTicketGroup = 32;
constexpr int kTicketLine = 32;  // uint32 words
constexpr int kTicketTop = kGradMaxBlocks / kTicketGroup;  // the groups' own counter
constexpr size_t kGradScratchBytes =
    (size_t)kGradMaxBlocks * 8 + (size_t)(kTicketTop + 1) * kTicketLine * 4;

// Sums of squares of one table's spans.  Slots [0, live) of `scratch` hold the
// sums of the tables before it, to which this one adds.  `norm` (the last
// table): the root of the sum of all slots goes there.  The tickets behind the
// slots are zero between calls.
hipError_t launch_grad_norm(const SpanTable<kNormSpans>& t, void* scratch, int live, int grid, float* norm,
                            hipStream_t s);
hipError_t launch_grad_clip(const SpanTable<kClipSpans>& t, const SpanOutputs& o, const float* norm,
                            float max_norm, int grid, hipStream_t s);
hipError_t launch_grad_clip(const SpanTable<kNormSpans>& t, const SpanShifts& o, const float* norm,
                            float max_norm, int grid, hipStream_t s);

// Tables of a list, one after the other (ar_ops.cpp).  ar_grad_norm's work.
int grad_norm_run(const ar_span_t* grads, size_t n, float* norm, void* scratch, hipStream_t s,
                  hipError_t* err);
// Argument checks of a norm, and its kernel arguments.  parts > 1: p.x is the
// reduce-scatter's send of that many rank rows of p.rows tokens each.
int norm_prepare(ar_rmsnorm_t p, int parts, NormArgs* out, bool* noop);

}  // namespace ar
