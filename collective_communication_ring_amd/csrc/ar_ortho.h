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
// 2^e and lo that of what is left, 22 significant bits of the two.  The host
// keeps e such that no value of the matrix passes 2^14; below it the bits of a
// value end at 2^-24, 2^-38 of the largest, so a matrix's error stays near
// 2^-23 of its norm however its values spread.  A row is cut into pieces of 32
// columns, 32 hi and then 32 lo: the 128 bytes that one row gives to one step
// of a product.  Columns are padded with zeros to whole pieces.
constexpr uint32_t kPiece = 32;
constexpr uint32_t padded(uint32_t n) { return (n + kPiece - 1) / kPiece * kPiece; }
constexpr int kOrthoTop = 14;

constexpr int kOrthoBatch = 128;  // matrices of one round of launches, at most
constexpr int kNormParts = 64;    // partial sums of a matrix's norm

struct OrthoPointers {
    const void* p[kOrthoBatch];
};

struct OrthoSplitArgs {
    double* parts;        // [count][kNormParts]
    _Float16* rowwise;    // [rows][2 padded(cols)], a matrix's `each` halves behind the last one's
    _Float16* colwise;    // [cols][2 padded(rows)]
    uint64_t each;
    uint64_t stride;      // of x
    uint32_t rows, cols;
    int bf16;
    float eps;
    double up;            // 2^e
};

// C = s_acc P Q^T + s_add D, P [m][K], Q [n][K], D and C [m][n], all in halves
// (s_acc and s_add hold the exponents too).
struct OrthoProductArgs {
    const _Float16 *p, *q, *d;  // d may be NULL
    _Float16* c;                // [m][2 padded(n)], or NULL
    _Float16* ct;               // [n][2 padded(m)], its transpose; or NULL
    uint64_t each_p, each_q, each_d, each_c, each_ct;  // from one matrix to the next
    uint32_t m, n, k;           // k: pieces
    int symmetric;              // C is (m == n, c == ct): tiles below the diagonal only, each
                                //   written to both its places
    float s_acc, s_add;
    // the last product: C goes to the caller's arrays instead, [m][n] or transposed
    int last, transposed, bf16;
    uint64_t out_stride;
};

hipError_t launch_ortho_split(const OrthoPointers& x, int count, const OrthoSplitArgs& a, hipStream_t s);
hipError_t launch_ortho_product(const OrthoPointers& out, int count, const OrthoProductArgs& a,
                                hipStream_t s);

}  // namespace ar
