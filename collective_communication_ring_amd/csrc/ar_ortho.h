// ar_ortho.h -- definitions shared by the host side (ar_ortho_host.cpp) and the HIP
// kernels (ar_ortho.hip) of the Newton-Schulz orthogonalisation.  Not part of
// the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ar.h"

namespace ar {

// A matrix in halves: value = (hi + lo) 2^-e, hi the nearest float16 of value
// 2^e and lo that of what is left: 22 significant bits of the two, off by 2^-23 of
// the value.  e is such that no value passes 2^14, by a bound of the matrix's
// singular values; the bits of a value end at 2^-24, so one below 2^-14 of the
// bound has fewer: it is off by 2^-39 of the bound.  Against the whole matrix's norm
// that is little; a row or column that is that much smaller than the others loses
// it for itself.
//
// The bound has two parts.  The host finds what X can reach, step by step, from a
// norm of 1.  A matrix whose norm is below eps starts further down, X in
// (2^-(t + 1), 2^-t], and t is found on the device: its arrays are kept 2^d
// higher, with d = max(0, t - h), h the powers of two by which the steps before can
// have brought X closer to the host's bound (OrthoLift).
//
// It is kept in pieces of 32 columns, piece by piece: 128 bytes a row, 32 hi and
// then 32 lo, all rows of a piece behind one another, so that what a tile's
// rows give to one step of a product is one stretch of memory.  (Row by row, the
// steps of a tile's rows lie at a distance that is often a power of two, all in
// one channel of an L2.)
// Columns are padded with zeros to whole pieces.
constexpr uint32_t kPiece = 32;
constexpr uint32_t padded(uint32_t n) { return (n + kPiece - 1) / kPiece * kPiece; }
constexpr int kOrthoTop = 14;

constexpr int kOrthoBatch = 128;  // matrices of one round of launches, at most
constexpr int kNormParts = 512;   // partial sums of a matrix's norm, at most; its t lies behind them

struct OrthoPointers {
    const void* p[kOrthoBatch];
};

// How far above the host's exponents a product's factors are for a matrix that
// starts 2^-t down: with n = max(0, t - now), m = max(0, t - next) and b = max(0, 2 n - b)
// the sums' factor gets 2^(acc . (n, m, b)), the addend's 2^(add . (n, m, b)).
struct OrthoLift {
    int now, next, b;
    int acc[3], add[3];
};
constexpr int kOrthoGround = 1 << 20;  // a `next` of the result: 0 whatever t
constexpr int kOrthoMostLift = 400;    // t at most: 2^-278 is the smallest float beside the largest eps

struct OrthoSplitArgs {
    double* parts;        // [count][kNormParts], of which nparts are in use (set by the launch)
    uint32_t nparts;
    _Float16* rowwise;    // x, a matrix's `each` halves behind the last one's
    _Float16* colwise;    // its transpose
    uint32_t* tickets;    // kOrthoTickets, zeroed
    uint64_t each;
    uint64_t stride;      // of x
    uint32_t rows, cols;
    int bf16;
    float eps;
    double up;            // 2^e
};

// C = s_acc P Q^T + s_add D + diag I, P [m][K], Q [n][K], all in halves (the
// factors hold the exponents too).
struct OrthoProductArgs {
    const _Float16 *p, *q;
    const _Float16* dt;         // D^T [n][m], or NULL
    _Float16 *c, *ct;           // C [m][n] and its transpose
    uint64_t each;              // from one matrix's arrays to the next one's
    uint32_t m, n, k;           // k: pieces
    int symmetric;              // C is (m == n, c == ct): tiles of the lower triangle only, each
                                //   written to both its places
    float s_acc, s_add, diag;
    OrthoLift lift;
    int ends;                   // a power of two that the last product's result gets besides
    const int* down;            // t of the first matrix, each / 2 ahead of the next one's
    // the last product: C goes to the caller's arrays instead, [m][n] or transposed
    int last, transposed, bf16;
    uint64_t out_stride;
    // few tiles: each by `parts` workgroups, a part of the pieces each (set by the launch)
    float* slots;               // [tile][part][its sums]
    uint32_t* tickets;          // a tile's, zero between launches
    uint32_t parts;
    uint32_t tiles_m, tiles_n, tiles;  // of a matrix, down and across, and all that are made
};

// Products whose tiles (of this side) go by parts, of so many pieces at least:
// workgroups and parts of a tile, at most; a slot holds a part's sums.
constexpr uint32_t kOrthoPartPieces = 16;
constexpr uint32_t kOrthoSlots = 256;
constexpr uint32_t kOrthoTickets = 256;
constexpr uint32_t kOrthoParts = 8;
constexpr uint32_t kOrthoPartTile = 64;
constexpr size_t kOrthoSlotBytes = kOrthoPartTile * kOrthoPartTile * 4;

// A small matrix goes through all its steps in one workgroup's LDS: X, its
// transpose, and one array for A and then B, whole 32 x 32 blocks of them, a block
// to each of 16 waves.
constexpr size_t kOrthoSmallBytes = 163584;  // and 256 bytes of sums: a CU's 160 KiB
inline bool ortho_small(uint32_t m, uint32_t n)
{
    const uint64_t mp = padded(m), np = padded(n);
    return mp * np <= 16 * 32 * 32 && (mp * np * 2 + mp * mp) * 4 <= kOrthoSmallBytes;
}

constexpr int kOrthoMaxSteps = 64;

struct OrthoSmallArgs {
    uint64_t x_stride, out_stride;
    uint32_t rows, cols;
    int bf16, steps;
    float eps;
    int ends;   // a power of two that the result gets besides
    double up;  // 2^e of the first X
    // a step's factors: A's, those of A A and A in B, of B X and X in X
    struct {
        float a, b_acc, b_add, x_acc, x_add;
    } step[kOrthoMaxSteps];
    short lift[kOrthoMaxSteps + 1];    // OrthoLift's now; the last: kOrthoSmallGround
    short lift_b[kOrthoMaxSteps];      // its b
};
constexpr int kOrthoSmallGround = 30000;

hipError_t launch_ortho_small(const OrthoPointers& x, const OrthoPointers& out, int count,
                              const OrthoSmallArgs& a, hipStream_t s);
hipError_t launch_ortho_split(const OrthoPointers& x, int count, const OrthoSplitArgs& a, hipStream_t s);
hipError_t launch_ortho_product(const OrthoPointers& out, int count, const OrthoProductArgs& a,
                                hipStream_t s);

}  // namespace ar
