// ar_ortho.hip -- kernels of the Newton-Schulz orthogonalisation: the norm, the
// split into halves, and their products.
//
//   X = x / (|x| + eps);  A = X X^T,  B = b A + c A A,  X = a X + B X
#include <algorithm>

#include "ar_norm_common.h"
#include "ar_ortho.h"

namespace ar {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;

__device__ inline float element(const void* p, uint64_t i, int bf16)
{
    return bf16 ? Elem<AR_BF16>::widen(static_cast<const uint16_t*>(p)[i])
                : static_cast<const float*>(p)[i];
}

// Sums of squares, 64-bit, of a matrix's rows in turn: [kNormParts] a matrix.
__global__ __launch_bounds__(kThreads) void k_ortho_norm(OrthoPointers x, OrthoSplitArgs a)
{
    __shared__ double s_f[kThreads / 64];
    const void* p = x.p[blockIdx.y];
    double sum = 0.0;
    for (uint32_t r = blockIdx.x; r < a.rows; r += kNormParts)
        for (uint32_t c = threadIdx.x; c < a.cols; c += kThreads) {
            const double v = (double)element(p, r * a.stride + c, a.bf16);
            sum += v * v;
        }
    sum = block_sum<kThreads / 64>(sum, s_f);
    if (threadIdx.x == 0)
        a.parts[blockIdx.y * (a.each / 4) + blockIdx.x] = sum;
}

__device__ inline void split(float v, _Float16* hi, _Float16* lo)
{
    *hi = (_Float16)v;
    *lo = (_Float16)(v - (float)*hi);
}

// Place of column c's hi half in a row.
__device__ inline uint32_t half_at(uint32_t c) { return c / kPiece * (2 * kPiece) + c % kPiece; }

// X in halves, rows and columns: tiles of 64 x 64, turned in LDS.
constexpr int kTile = 64;
__global__ __launch_bounds__(kThreads) void k_ortho_split(OrthoPointers x, OrthoSplitArgs a)
{
    __shared__ float s_t[kTile][kTile + 1];
    __shared__ double s_up;
    const void* p = x.p[blockIdx.z];
    if (threadIdx.x < 64) {
        const double sum = wave_sum(a.parts[blockIdx.z * (a.each / 4) + threadIdx.x]);
        if (threadIdx.x == 0)
            s_up = a.up / (sqrt(sum) + (double)a.eps);
    }
    __syncthreads();
    const uint32_t r0 = blockIdx.y * kTile, c0 = blockIdx.x * kTile;
    const uint32_t i = threadIdx.x % kTile, j0 = threadIdx.x / kTile;
    const uint64_t at = blockIdx.z * a.each;
    const uint32_t cols = padded(a.cols), rows = padded(a.rows);
    for (uint32_t j = j0; j < kTile; j += kThreads / kTile) {
        const uint32_t r = r0 + j, c = c0 + i;
        float v = 0.0f;
        if (r < a.rows && c < a.cols)
            v = (float)((double)element(p, r * a.stride + c, a.bf16) * s_up);
        s_t[j][i] = v;
        if (r < a.rows && c < cols) {
            _Float16* o = a.rowwise + at + (uint64_t)r * 2 * cols + half_at(c);
            split(v, o, o + kPiece);
        }
    }
    __syncthreads();
    for (uint32_t j = j0; j < kTile; j += kThreads / kTile) {
        const uint32_t c = c0 + j, r = r0 + i;
        if (c < a.cols && r < rows) {
            _Float16* o = a.colwise + at + (uint64_t)c * 2 * rows + half_at(r);
            split(s_t[i][j], o, o + kPiece);
        }
    }
}

__device__ inline void copy16(const void* from, void* to_wave)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)from,
                                     (__attribute__((address_space(3))) uint32_t*)to_wave, 16, 0, 0);
}

// Rows [row0, row0 + ROWS) of a piece to LDS, 128 bytes a row; rows past the
// last are the last.  Chunk c (16 bytes) of row r lies at r * 8 + (c ^ r % 8),
// so that eight rows' same chunk, as the matrix instructions take it, are in
// different banks.
template <int ROWS, int WAVES>
__device__ inline void stage(const _Float16* p, uint32_t row0, uint32_t rows, uint64_t stride,
                             _Float16* lds, uint32_t wave, uint32_t lane)
{
#pragma unroll
    for (int i = 0; i < ROWS / 8 / WAVES; ++i) {
        const uint32_t r = (i * WAVES + wave) * 8 + lane / 8;
        const uint32_t row = row0 + r < rows ? row0 + r : rows - 1;
        copy16(p + row * stride + ((lane % 8) ^ (r % 8)) * 8,
               lds + (i * WAVES + wave) * 8 * 2 * kPiece);
    }
}

// C = s_acc P Q^T + s_add D by tiles of BM x BN, a wave WM x WN of them in 32 x
// 32 products: hi hi + hi lo + lo hi for each 32 columns (lo lo is below 2^-22
// of their product).
template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void k_ortho_product(OrthoPointers out,
                                                                              OrthoProductArgs a)
{
    constexpr int WAVES = (BM / WM) * (BN / WN), TM = WM / 32, TN = WN / 32;
    __shared__ _Float16 s_p[2][BM * 2 * kPiece], s_q[2][BN * 2 * kPiece];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    uint32_t ti = blockIdx.x, tj = blockIdx.y;
    if (a.symmetric) {  // tile number blockIdx.x of the lower triangle, row by row
        ti = (uint32_t)((sqrtf(8.0f * (float)blockIdx.x + 1.0f) - 1.0f) * 0.5f);
        while (ti * (ti + 1) / 2 > blockIdx.x)
            --ti;
        while ((ti + 1) * (ti + 2) / 2 <= blockIdx.x)
            ++ti;
        tj = blockIdx.x - ti * (ti + 1) / 2;
    }
    const uint32_t i0 = ti * BM, j0 = tj * BN;
    const uint64_t stride = (uint64_t)a.k * 2 * kPiece;
    const _Float16* p = a.p + blockIdx.z * a.each_p;
    const _Float16* q = a.q + blockIdx.z * a.each_q;
    const uint32_t wi = wave / (BN / WN) * WM, wj = wave % (BN / WN) * WN;

    f32x16 acc[TM][TN];
#pragma unroll
    for (int x = 0; x < TM; ++x)
#pragma unroll
        for (int y = 0; y < TN; ++y)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[x][y][i] = 0.0f;

    stage<BM, WAVES>(p, i0, a.m, stride, s_p[0], wave, lane);
    stage<BN, WAVES>(q, j0, a.n, stride, s_q[0], wave, lane);
    for (uint32_t k = 0; k < a.k; ++k) {
        __syncthreads();  // this piece is there, and nobody reads the other one
        if (k + 1 < a.k) {
            stage<BM, WAVES>(p + (k + 1) * 2 * kPiece, i0, a.m, stride, s_p[(k + 1) & 1], wave, lane);
            stage<BN, WAVES>(q + (k + 1) * 2 * kPiece, j0, a.n, stride, s_q[(k + 1) & 1], wave, lane);
        }
        const _Float16 *sp = s_p[k & 1], *sq = s_q[k & 1];
        const auto part = [&](const _Float16* s, uint32_t row, uint32_t chunk) {
            return *reinterpret_cast<const f16x8*>(s + (row * 8 + (chunk ^ row % 8)) * 8);
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 16 columns
            const uint32_t chunk = 2 * h + lane / 32;
            f16x8 ph[TM], pl[TM], qh[TN], ql[TN];
#pragma unroll
            for (int x = 0; x < TM; ++x) {
                ph[x] = part(sp, wi + x * 32 + lane % 32, chunk);
                pl[x] = part(sp, wi + x * 32 + lane % 32, chunk + 4);
            }
#pragma unroll
            for (int y = 0; y < TN; ++y) {
                qh[y] = part(sq, wj + y * 32 + lane % 32, chunk);
                ql[y] = part(sq, wj + y * 32 + lane % 32, chunk + 4);
            }
#pragma unroll
            for (int x = 0; x < TM; ++x)
#pragma unroll
                for (int y = 0; y < TN; ++y) {
                    acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl[x], qh[y], acc[x][y], 0, 0, 0);
                    acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[x], ql[y], acc[x][y], 0, 0, 0);
                    acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph[x], qh[y], acc[x][y], 0, 0, 0);
                }
        }
    }

    // lane l holds column l % 32, rows 8 (r / 4) + 4 (l / 32) + r % 4 of a 32 x 32 product
    const uint32_t mp = padded(a.m), np = padded(a.n);
    const _Float16* d = a.d ? a.d + blockIdx.z * a.each_d : nullptr;
    _Float16* c = a.c + blockIdx.z * a.each_c;
    _Float16* ct = a.ct + blockIdx.z * a.each_ct;
    void* to = const_cast<void*>(out.p[blockIdx.z]);
#pragma unroll
    for (int x = 0; x < TM; ++x)
#pragma unroll
        for (int y = 0; y < TN; ++y) {
            const uint32_t j = j0 + wj + y * 32 + lane % 32;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t i = i0 + wi + x * 32 + 8 * g + 4 * (lane / 32);
                f16x4 hi, lo;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float v = 0.0f;
                    if (i + r < a.m && j < a.n) {
                        v = acc[x][y][4 * g + r] * a.s_acc;
                        if (d) {
                            const _Float16* e = d + (uint64_t)(i + r) * 2 * np + half_at(j);
                            v = fmaf((float)e[0] + (float)e[kPiece], a.s_add, v);
                        }
                    }
                    _Float16 vh, vl;
                    split(v, &vh, &vl);
                    hi[r] = vh;
                    lo[r] = vl;
                    if (a.last) {
                        if (i + r < a.m && j < a.n) {
                            const uint64_t at = a.transposed ? j * a.out_stride + (i + r)
                                                             : (i + r) * a.out_stride + j;
                            if (a.bf16)
                                static_cast<uint16_t*>(to)[at] = Elem<AR_BF16>::narrow(v);
                            else
                                static_cast<float*>(to)[at] = v;
                        }
                    } else if (i + r < a.m && j < np) {
                        _Float16* o = c + (uint64_t)(i + r) * 2 * np + half_at(j);
                        o[0] = vh;
                        o[kPiece] = vl;
                    }
                }
                if (!a.last && (!a.symmetric || ti != tj) && j < a.n && i < mp) {
                    _Float16* o = ct + (uint64_t)j * 2 * mp + half_at(i);
                    *reinterpret_cast<f16x4*>(o) = hi;
                    *reinterpret_cast<f16x4*>(o + kPiece) = lo;
                }
            }
        }
}

}  // namespace

hipError_t launch_ortho_split(const OrthoPointers& x, int count, const OrthoSplitArgs& a, hipStream_t s)
{
    hipLaunchKernelGGL(k_ortho_norm, dim3(kNormParts, count), dim3(kThreads), 0, s, x, a);
    hipLaunchKernelGGL(k_ortho_split,
                       dim3((padded(a.cols) + kTile - 1) / kTile, (padded(a.rows) + kTile - 1) / kTile,
                            count),
                       dim3(kThreads), 0, s, x, a);
    return hipGetLastError();
}

hipError_t launch_ortho_product(const OrthoPointers& out, int count, const OrthoProductArgs& a,
                                hipStream_t s)
{
    constexpr int B = 128;
    const uint32_t ti = (a.m + B - 1) / B, tj = (a.n + B - 1) / B;
    const dim3 grid = a.symmetric ? dim3(ti * (ti + 1) / 2, 1, count) : dim3(ti, tj, count);
    hipLaunchKernelGGL((k_ortho_product<B, B, 64, 64>), grid, dim3(256), 0, s, out, a);
    return hipGetLastError();
}

}  // namespace ar
