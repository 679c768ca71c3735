// ar_heads.h -- definitions shared by the host side (ar_heads_host.cpp) and the HIP
// kernels of the operators on attention heads: rotation and head norm
// (ar_heads.hip), the norm's backward pass (ar_heads_back.hip).  Not part of
// the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ar.h"

namespace ar {

// Division of numbers below 2^31 by a fixed one: n d^-1 is n mul >> shift, mul
// = floor(2^(31 + l) / d) + 1 with 2^l >= d, whose excess over the quotient is
// below n / 2^(31 + l) < 1 / d.
struct FastDiv {
    uint32_t by, mul, shift;
};
inline FastDiv fast_div(uint32_t d)
{
    uint32_t l = 0;
    while (((uint64_t)1 << l) < d)
        ++l;
    return {d, (uint32_t)(((uint64_t)1 << (31 + l)) / d + 1), 31 + l};
}

// Distances of an array of heads, in elements.
struct HeadsArray {
    void* p;
    uint64_t batch, token, head;
};

// The rotation, as kernels take it.
struct Turn {
    const double* frequencies;
    const void* positions;
    uint64_t position_stride;
    int wide;        // positions are 64-bit
    int layout;
    uint32_t pairs;  // rot_dim / 2
    uint32_t slots;  // pairs, rounded up to a vector's: the length of a token's table
    float factor;
    float sign;      // -1: the transpose
    FastDiv per_slot;
};

struct HeadsArgs {
    HeadsArray x[2], y[2];  // queries, keys
    const void* weight[2];  // the norm only
    uint32_t heads0;        // of the queries
    uint32_t rows;          // batch * tokens * heads
    FastDiv heads, tokens;  // of a token (both sides); of a batch
    uint32_t dim, nvec;     // elements and vectors of a head
    uint32_t turned;        // units that are rotated
    uint32_t lanes;         // threads per head
    uint32_t turns;         // heads a group of lanes takes, one after the other
    float eps;
    int weight_f32;
    int stream;             // outputs larger than the L2s
    Turn turn;
};

struct HeadsBackArgs {
    HeadsArray dy[2], x[2], dx[2];
    const void* weight[2];
    float* dweight[2];      // [ranks][dim]
    float* partial;         // [ranks][blocks of both sides][dim]
    uint32_t heads[2];
    FastDiv head[2];        // division by heads
    FastDiv tokens;
    uint32_t rows[2];       // of one rank: heads of its batches
    uint32_t rank_tokens;   // tokens of one rank, all its batches
    uint32_t dim, nvec;
    uint32_t turned;
    uint32_t lanes;
    int ranks;
    int blocks[2];          // workgroups per rank
    float eps;
    int weight_f32;
    int stream;
    Turn turn;
};

constexpr uint32_t kHeadMaxDim = 1024;
constexpr int kHeadPerLane = 16;  // elements of a head that a thread holds

// Partial rows of the weights' gradients of all ranks and both sides, at most
// (a rank has one at least for each side).
constexpr int kHeadBackBlocks = 1024;
inline int head_back_blocks(int ranks)
{
    const int b = kHeadBackBlocks / ranks;
    return b < 2 ? 2 : b;
}

// Elements of a vector: the widest of 16 bytes and less that divides a head,
// and in the layout of halves the half that is rotated.
int heads_vector(int dtype, uint32_t dim, const Turn& t);
// The fields that follow from it.
void heads_fit(uint32_t dim, int w, uint32_t* nvec, uint32_t* turned, uint32_t* lanes, Turn* t);

hipError_t launch_heads(int dtype, bool norm, HeadsArgs a, hipStream_t s);
hipError_t launch_heads_back(int dtype, HeadsBackArgs a, hipStream_t s);

}  // namespace ar
