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
    uint32_t pairs;  // rot_dim / 2: 0 for no rotation
    float factor;
    float sign;      // -1: the transpose
    uint32_t lanes;  // that take a token's pairs: a power of two, 64 at most
};

struct HeadsArgs {
    HeadsArray x[2], y[2];  // queries, keys
    const void* weight[2];  // the norm only
    uint32_t heads0;        // of the queries
    uint32_t rows;          // batch * tokens * heads
    uint32_t first;         // workgroup of the launch (set by it)
    FastDiv heads, tokens;  // of a token (both sides); of a batch
    uint32_t dim, nvec;     // elements and vectors of a head
    uint32_t turned;        // rotated units of a head, halves
    uint32_t lanes;         // threads per head
    uint32_t turns;         // heads a group of lanes takes, one after the other
    uint32_t table;         // cosines and sines of a wave's tokens, at most
    float eps, per_dim;     // per_dim: 1 / dim
    int weight_f32;
    int stream;             // outputs larger than the L2s
    Turn turn;
};

// How a thread goes from one of its heads to the next: so many heads and tokens
// on, or one token more where that passes a token's last head.
struct HeadsStep {
    uint32_t heads, tokens;
    // elements that x, dy and dx are moved by, and further by with that token
    uint64_t by[3], more[3];
};

struct HeadsBackArgs {
    HeadsArray dy[2], x[2], dx[2];
    HeadsStep step[2];      // (set by the launch)
    const void* weight[2];
    float* dweight[2];      // [ranks][dim]
    float* partial;         // [ranks][blocks][both sides][dim]
    uint32_t heads[2];
    FastDiv head[2];        // division by heads
    FastDiv tokens;
    uint32_t rank_batches, rank_tokens;  // of one rank: batches, and tokens of all of them
    uint32_t dim, nvec;
    uint32_t turned;
    uint32_t lanes;
    int ranks;
    uint32_t blocks;        // workgroups per rank
    uint32_t chunk;         // tokens whose angles are made at once, of one batch
    uint32_t batch_chunks;  // chunks of a batch
    uint32_t run;           // chunks of a wave
    int apart;              // waves have queries and keys in turn, of one chunk
    FastDiv chunks;         // division by batch_chunks
    float eps, per_dim;
    int weight_f32;
    int stream;
    Turn turn;
};

constexpr uint32_t kHeadMaxDim = 1024;
constexpr uint32_t kHeadsMostBlocks = 1u << 23;  // of a launch: a grid has less than 2^32 threads
constexpr int kHeadPerLane = 16;  // elements of a head that a thread holds

// Workgroups of the backward pass, at most; each leaves a partial row of both weights'
// gradients.  Three on each CU, which the forms of bfloat16 vectors of 16 bytes reach
// (146 to 154 registers).  The others have 172 to 234 and two on a CU, for which the
// most is a round and a half (float32, 16384 x (16 + 4) heads of 128: 97 us, 5.2 TB/s).
constexpr int kHeadBackBlocks = 768;
inline int head_back_blocks(int ranks) { return kHeadBackBlocks / ranks; }

// LDS of the backward pass, in bytes: both weights at 0, from `sums` on the sums of
// the side that a wave is not at (read 16 bytes at a time), from `angles` on the
// waves' angles; at the end, from 0 on, a partial row of each wave.
struct HeadBackPlaces {
    uint32_t sums, angles, bytes;
};
inline __host__ __device__ HeadBackPlaces head_back_places(uint32_t dim, uint32_t threads, uint32_t waves,
                                                           uint32_t wave_angles)
{
    HeadBackPlaces p;
    p.sums = (dim + 1) / 2 * 16;
    p.angles = p.sums + threads * kHeadPerLane * 4;
    p.bytes = p.angles + waves * wave_angles * 8;
    const uint32_t rows = waves * dim * 4;
    p.bytes = p.bytes < rows ? rows : p.bytes;
    return p;
}

// Elements of a vector: the widest of 16 bytes and less that divides a head,
// and in the layout of halves the half that is rotated.
int heads_vector(int dtype, uint32_t dim, const Turn& t);
// The fields that follow from it.
void heads_fit(uint32_t dim, int w, uint32_t* nvec, uint32_t* turned, uint32_t* lanes, Turn* t);

hipError_t launch_heads(int dtype, bool norm, HeadsArgs a, hipStream_t s);
hipError_t launch_heads_back(int dtype, HeadsBackArgs a, hipStream_t s);

}  // namespace ar
