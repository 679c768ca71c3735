// ar_ortho.hip -- kernels of the Newton-Schulz orthogonalisation: the norm, the
// split into halves, and their products.
//
//   X = x / (|x| + eps);  A = X X^T,  B = b A + c A A,  X = a X + B X
#include <algorithm>
#include <utility>

#include "ar_norm_common.h"
#include "ar_ortho.h"

namespace ar {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;

// Sums of squares, 64-bit, of a matrix's vectors in turn: [parts] a matrix.
// Zeroes the tickets, too.
template <class E>
__global__ __launch_bounds__(kThreads) void k_ortho_norm(OrthoPointers x, OrthoSplitArgs a)
{
    __shared__ double s_f[kThreads / 64];
    const typename E::T* p = static_cast<const typename E::T*>(x.p[blockIdx.y]);
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (uint32_t i = threadIdx.x; i < kOrthoTickets; i += kThreads)
            a.tickets[i] = 0;
    double sum = 0.0;
    if (a.cols < E::VEC) {
        for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < a.rows * a.cols; i += gridDim.x * kThreads) {
            const double v = E::widen(p[i / a.cols * a.stride + i % a.cols]);
            sum = fma(v, v, sum);
        }
    } else {
        const uint32_t vecs = (a.cols + E::VEC - 1) / E::VEC, all = a.rows * vecs;
        for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < all; i += gridDim.x * kThreads) {
            const uint32_t r = i / vecs, c = (i - r * vecs) * E::VEC;
            u32x4 raw = load_vec<E>(p + r * a.stride, c, a.cols);
            fit<E>(raw, c, a.cols);
            float v[E::VEC];
            widen_slot<E, E::VEC>(raw, v);
#pragma unroll
            for (int k = 0; k < E::VEC; ++k)
                sum = fma((double)v[k], (double)v[k], sum);
        }
    }
    sum = block_sum<kThreads / 64>(sum, s_f);
    if (threadIdx.x == 0)
        a.parts[blockIdx.y * (a.each / 4) + blockIdx.x] = sum;
}

// t of a matrix whose X has this norm (OrthoLift): 0 for one near 1, and for zeros
// and what is no number.
__device__ inline int down_of(double norm)
{
    if (!(norm > 0.0 && norm < 0.5))
        return 0;
    const int t = -__builtin_amdgcn_frexp_exp(norm);
    return t < kOrthoMostLift ? t : kOrthoMostLift;
}

__device__ inline int above(int v) { return v > 0 ? v : 0; }

// How much of a last product's power of two its result gets in the end: half of a
// large one, as a factor that is subnormal has fewer bits.
__device__ inline int halved_end(int power) { return power < -32 ? power / 2 : 0; }

__device__ inline void split(float v, _Float16* hi, _Float16* lo)
{
    *hi = (_Float16)v;
    *lo = (_Float16)(v - (float)*hi);
}

// Place of the hi half of (r, c) in a matrix of `rows` rows; the lo half is
// kPiece behind it.
__device__ inline uint64_t half_at(uint32_t r, uint32_t c, uint32_t rows)
{
    return ((uint64_t)(c / kPiece) * rows + r) * (2 * kPiece) + c % kPiece;
}

// Eight consecutive columns of a row in halves.
__device__ inline void store_halves(_Float16* o, const float (&v)[8])
{
    f16x8 hi, lo;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        _Float16 h, l;
        split(v[i], &h, &l);
        hi[i] = h;
        lo[i] = l;
    }
    *reinterpret_cast<f16x8*>(o) = hi;
    *reinterpret_cast<f16x8*>(o + kPiece) = lo;
}

// X in halves, rows and columns: tiles of 64 x 64, turned in LDS, eight columns
// (rows) of a row (column) a thread.
constexpr int kTile = 64;
template <class E>
__global__ __launch_bounds__(kThreads) void k_ortho_split(OrthoPointers x, OrthoSplitArgs a)
{
    __shared__ float s_t[kTile][kTile + 1];
    __shared__ double s_up;
    const typename E::T* p = static_cast<const typename E::T*>(x.p[blockIdx.z]);
    if (threadIdx.x < 64) {
        double sum = 0.0;
        for (uint32_t i = threadIdx.x; i < a.nparts; i += 64)
            sum += a.parts[blockIdx.z * (a.each / 4) + i];
        const double norm = sqrt(wave_sum(sum));
        if (threadIdx.x == 0) {
            const double by = norm + (double)a.eps;
            const int down = down_of(norm / by);
            s_up = ldexp(a.up, down) / by;
            if (blockIdx.x == 0 && blockIdx.y == 0)
                *reinterpret_cast<int*>(a.parts + blockIdx.z * (a.each / 4) + kNormParts) = down;
        }
    }
    const uint32_t r0 = blockIdx.y * kTile, c0 = blockIdx.x * kTile;
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t r = r0 + h * 32 + threadIdx.x / 8, c = c0 + threadIdx.x % 8 * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[h][i] = 0.0f;
        if (r >= a.rows)
            continue;
        const typename E::T* row = p + r * a.stride;
        if (c + 8 <= a.cols) {
#pragma unroll
            for (int g = 0; g < 8; g += E::VEC) {
                float w[E::VEC];
                widen_slot<E, E::VEC>(load_vec<E>(row, c + g, a.cols), w);
#pragma unroll
                for (int i = 0; i < E::VEC; ++i)
                    v[h][g + i] = w[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < a.cols)
                    v[h][i] = E::widen(row[c + i]);
        }
    }
    __syncthreads();
    const double up = s_up;
    const uint64_t at = blockIdx.z * a.each;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t j = h * 32 + threadIdx.x / 8, i0 = threadIdx.x % 8 * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[h][i] = (float)((double)v[h][i] * up);
            s_t[j][i0 + i] = v[h][i];
        }
        if (r0 + j < a.rows && c0 + i0 < padded(a.cols))
            store_halves(a.rowwise + at + half_at(r0 + j, c0 + i0, a.rows), v[h]);
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t j = threadIdx.x % 64, i0 = (h * 4 + threadIdx.x / 64) * 8;
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = s_t[i0 + i][j];
        if (c0 + j < a.cols && r0 + i0 < padded(a.rows))
            store_halves(a.colwise + at + half_at(c0 + j, r0 + i0, a.cols), w);
    }
}

// f(0), f(1), ... f(N - 1), of constants.
template <class F, int... I>
__device__ inline void each_of(F f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ inline void each_of(F f)
{
    each_of(f, std::make_integer_sequence<int, N>{});
}

// Copies 16 bytes a lane to LDS, at `to` (an address there) for the wave's first
// lane and on.  Written out, as the compiler would wait for all such copies ahead
// of any read of LDS; they have no result, and what they move is waited for by
// wait_and_meet.  (m0 holds the address; its writing takes a cycle.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is nobody's here
__device__ inline void copy16(const void* from, uint32_t to)
{
    __asm__ __volatile__("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from)
                         : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ inline uint32_t lds_address(const void* p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// The element rows of a piece that a thread copies to LDS, 16 bytes each.  Row r
// of the tile has 128 bytes there, its chunk c of 16 at r * 8 + (c ^ r / 2 % 8),
// so that 16 rows' same chunk, as the matrix instructions take it, are in all 64
// banks; rows past the matrix's last are the last.
template <int ROWS, int WAVES>
struct Stage {
    static constexpr int N = ROWS / 8 / WAVES;
    uint32_t at[N];  // bytes into the piece
    __device__ void set(uint32_t row0, uint32_t rows, uint32_t wave, uint32_t lane)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t r = (i * WAVES + wave) * 8 + lane / 8;
            const uint32_t row = row0 + r < rows ? row0 + r : rows - 1;
            at[i] = row * (4 * kPiece) + ((lane % 8) ^ (r / 2 % 8)) * 16;
        }
    }
    template <int I>
    __device__ void copy(const char* piece, uint32_t lds, uint32_t wave) const
    {
        copy16(piece + at[I], lds + (I * WAVES + wave) * (8 * 4 * kPiece));
    }
};

// The 4 x 4 words of four neighbouring lanes' w[0 .. 3], transposed.
__device__ inline void transpose4(uint32_t (&w)[4])
{
    const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
#pragma unroll
    for (int r = 0; r < 4; r += 2) {
        const uint32_t got = dpp<kXor1>(odd ? w[r] : w[r + 1]);
        w[r] = odd ? got : w[r];
        w[r + 1] = odd ? w[r + 1] : got;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const uint32_t got = dpp<kXor2>(high ? w[r] : w[r + 2]);
        w[r] = high ? got : w[r];
        w[r + 2] = high ? w[r + 2] : got;
    }
}

// Four values, or the first n of them, to the caller's array.
__device__ inline void store_out(void* to, int bf16, uint64_t at, uint32_t n, const float (&v)[4])
{
    if (bf16) {
        uint16_t* o = static_cast<uint16_t*>(to) + at;
        if (n >= 4) {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2), aligned(2)));
            typedef float f32x4 __attribute__((ext_vector_type(4)));
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            const f32x4 f = {v[0], v[1], v[2], v[3]};
            *reinterpret_cast<u32x2*>(o) = __builtin_bit_cast(u32x2, __builtin_convertvector(f, bf16x4));
        } else {
#pragma unroll
            for (uint32_t r = 0; r < 3; ++r)
                if (r < n)
                    o[r] = Elem<AR_BF16>::narrow(v[r]);
        }
    } else {
        float* o = static_cast<float*>(to) + at;
        if (n >= 4) {
            *reinterpret_cast<typename AnyVec<float>::type*>(o) =
                u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3])};
        } else {
#pragma unroll
            for (uint32_t r = 0; r < 3; ++r)
                if (r < n)
                    o[r] = v[r];
        }
    }
}

// C = s_acc P Q^T + s_add D + diag I by tiles of B x B, a wave WM x WN of them in 32 x
// 32 products: lo hi + hi lo + hi hi for each 32 columns (lo lo is below 2^-22
// of their product).  While a piece is multiplied, the next S - 1 are on their
// way to LDS, by copies that need no registers.
template <int B, int WM, int WN>
struct Product {
    static constexpr int WAVES = (B / WM) * (B / WN), TM = WM / 32, TN = WN / 32;
    static constexpr int COPIES = 2 * B / 8 / WAVES;  // of a thread, a piece
    static constexpr int STAGE = 2 * B * 2 * kPiece;  // halves of LDS, a piece
    f32x16 acc[TM][TN];
    Stage<B, WAVES> sp;
    Stage<B, WAVES> sq;
    const char *p, *q;  // the next piece to copy
    uint64_t step_p, step_q;

    // The I-th of a thread's copies of the next piece, to `to`.
    template <int I>
    __device__ void copy(uint32_t to, uint32_t wave) const
    {
        if constexpr (I < B / 8 / WAVES)
            sp.template copy<I>(p, to, wave);
        else
            sq.template copy<I - B / 8 / WAVES>(q, to + B * 4 * kPiece, wave);
    }
    // To the next piece, if there is one: the last is copied again otherwise (and
    // not used), so that all turns of the loop are alike.
    __device__ void advance(bool more)
    {
        p += more ? step_p : 0;
        q += more ? step_q : 0;
    }

    // What a lane multiplies of 16 columns: row lane % 32 of each 32, 8 columns.
    static constexpr int READS = 2 * (TM + TN);
    struct Part {
        f16x8 ph[TM], pl[TM], qh[TN], ql[TN];
    };
    // The I-th read of LDS for the H-th 16 columns of the piece at s.
    template <int I, int H>
    static __device__ void read(Part* o, const _Float16* s, uint32_t wi, uint32_t wj, uint32_t lane)
    {
        constexpr int t = I / 2;
        const uint32_t row = lane % 32, chunk = 2 * H + lane / 32 + (I % 2 ? 0 : 4);
        const uint32_t first = t < TM ? wi + t * 32 : B + wj + (t - TM) * 32;
        const f16x8 v = *reinterpret_cast<const f16x8*>(s + (first + row) * (2 * kPiece) +
                                                        (chunk ^ row / 2 % 8) * 8);
        if constexpr (t < TM)
            (I % 2 ? o->ph[t] : o->pl[t]) = v;
        else
            (I % 2 ? o->qh[t - TM] : o->ql[t - TM]) = v;
    }

    // The products of 16 columns; between(n) after the n-th of MULTIPLIES: what else
    // the wave issues goes there, one by one, as the matrix pipe has work for 32
    // cycles then, and a run of copies or reads would hold up the wave for as long
    // as its queue takes.
    static constexpr int MULTIPLIES = 3 * TM * TN;
    template <class F>
    __device__ void multiply(const Part& o, F between)
    {
        each_of<MULTIPLIES>([&](auto number) {
            constexpr int n = number.value, x = n / TN % TM, y = n % TN, term = n / (TM * TN);
            acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(term == 0 ? o.pl[x] : o.ph[x],
                                                               term == 1 ? o.ql[y] : o.qh[y],
                                                               acc[x][y], 0, 0, 0);
            between(number);
            __builtin_amdgcn_sched_barrier(0);
        });
    }
};

// What a thread waits for until at most N of its copies are on their way, and
// then everyone: the pieces before those are in LDS, and what was read there has
// been.
template <int N>
__device__ inline void wait_and_meet()
{
    __asm__ __volatile__("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | N >> 4 << 14);  // vmcnt(N) lgkmcnt(0)
    __asm__ __volatile__("s_barrier" ::: "memory");
}

// Workgroups go round the 8 XCDs; this numbers them such that each XCD has a
// run of numbers, whose tiles share rows in its L2.
__device__ inline uint32_t xcd_block(uint32_t b, uint32_t of)
{
    const uint32_t xcd = b % 8, each = of / 8, more = of % 8;
    return xcd * each + (xcd < more ? xcd : more) + b / 8;
}

// Tile of a number: bands of 8 rows of tiles, column by column; of a symmetric
// product the lower triangle.
__device__ inline void place_tile(uint32_t t, const OrthoProductArgs& a, uint32_t* ti, uint32_t* tj)
{
    constexpr uint32_t B = 8;
    if (a.symmetric) {
        uint32_t r = (uint32_t)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
        while (r * (r + 1) / 2 > t)
            --r;
        while ((r + 1) * (r + 2) / 2 <= t)
            ++r;
        const uint32_t first = r / B * B;  // of the band; below it are first (first + 1) / 2 tiles
        const uint32_t rows = a.tiles_m - first < B ? a.tiles_m - first : B;
        t -= first * (first + 1) / 2;
        if (t < first * rows) {
            *tj = t / rows;
            *ti = first + t % rows;
        } else {  // the triangle at its end
            t -= first * rows;
            uint32_t i = 0;
            for (; (i + 1) * (i + 2) / 2 <= t; ++i)
                ;
            *ti = first + i;
            *tj = first + t - i * (i + 1) / 2;
        }
    } else {
        const uint32_t first = t / (B * a.tiles_n) * B;
        const uint32_t rows = a.tiles_m - first < B ? a.tiles_m - first : B;
        t -= first * a.tiles_n;
        *tj = t / rows;
        *ti = first + t % rows;
    }
}

template <int B, int WM, int WN, int S, bool PARTS>
__global__ __launch_bounds__(64 * (B / WM) * (B / WN)) void k_ortho_product(OrthoPointers out,
                                                                              OrthoProductArgs a)
{
    using P = Product<B, WM, WN>;
    constexpr int TM = P::TM, TN = P::TN, THREADS = 64 * P::WAVES;
    __shared__ __attribute__((aligned(16))) _Float16 s_piece[S * P::STAGE];
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    uint32_t tile = xcd_block(blockIdx.x, gridDim.x), part = 0;
    if constexpr (PARTS) {
        part = tile % a.parts;
        tile /= a.parts;
    }
    const uint32_t number = tile, matrix = tile / a.tiles;
    tile -= matrix * a.tiles;
    uint32_t ti, tj;
    place_tile(tile, a, &ti, &tj);
    const uint32_t i0 = ti * B, j0 = tj * B;
    const uint32_t wi = wave / (B / WN) * WM, wj = wave % (B / WN) * WN;
    const uint64_t own = matrix * a.each;
    uint32_t k0 = 0, k1 = a.k;
    if constexpr (PARTS) {
        k0 = a.k * part / a.parts;
        k1 = a.k * (part + 1) / a.parts;
    }

    P g;
#pragma unroll
    for (int x = 0; x < TM; ++x)
#pragma unroll
        for (int y = 0; y < TN; ++y)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                g.acc[x][y][i] = 0.0f;
    g.sp.set(i0, a.m, wave, lane);
    g.sq.set(j0, a.n, wave, lane);
    g.step_p = (uint64_t)a.m * (4 * kPiece);
    g.step_q = (uint64_t)a.n * (4 * kPiece);
    g.p = reinterpret_cast<const char*>(a.p + own) + k0 * g.step_p;
    g.q = reinterpret_cast<const char*>(a.q + own) + k0 * g.step_q;
    // in registers by now: a load of them on its way would have the loop wait for
    // all of its reads of LDS
    void* to = const_cast<void*>(out.p[matrix]);
    const int down = a.down[matrix * (a.each / 2)];
    __asm__ __volatile__("" ::"s"(to), "s"(a.out_stride), "s"(down));
    const uint32_t lds = lds_address(s_piece);
#pragma unroll
    for (uint32_t o = 0; o < S; ++o) {
        each_of<P::COPIES>([&](auto i) { g.template copy<i.value>(lds + o * (P::STAGE * 2), wave); });
        g.advance(k0 + o + 1 < k1);
    }
    wait_and_meet<(S - 1) * P::COPIES>();
    typename P::Part first, second;  // of a piece, 16 columns each
    each_of<P::READS>([&](auto i) { P::template read<i.value, 0>(&first, s_piece, wi, wj, lane); });
    uint32_t at = 0;
    for (uint32_t k = k0; k < k1; ++k) {
        const _Float16* here = s_piece + at * P::STAGE;
        const uint32_t free = lds + at * (P::STAGE * 2);
        at = at + 1 == S ? 0 : at + 1;
        const _Float16* next = s_piece + at * P::STAGE;
        __builtin_amdgcn_sched_barrier(0);
        g.multiply(first, [&](auto n) {
            constexpr int each = P::MULTIPLIES > P::READS ? 1 : 2;
            each_of<each>([&](auto o) {
                constexpr int i = n.value * each + o.value;
                if constexpr (i < P::READS)
                    P::template read<i, 1>(&second, here, wi, wj, lane);
            });
        });
        // the next piece is there, and everybody has read this one: its place is free
        wait_and_meet<(S - 2) * P::COPIES>();
        g.multiply(second, [&](auto n) {
            constexpr int all = P::READS + P::COPIES;
            constexpr int each = (all + P::MULTIPLIES - 1) / P::MULTIPLIES;
            each_of<each>([&](auto o) {
                constexpr int i = n.value * each + o.value;
                if constexpr (i < P::READS)
                    P::template read<i, 0>(&first, next, wi, wj, lane);
                else if constexpr (i < all)
                    g.template copy<i - P::READS>(free, wave);
            });
        });
        g.advance(k + S + 1 < k1);
    }
    wait_and_meet<0>();  // no copy may be on its way when the workgroup ends

    if constexpr (PARTS) {
        // A part's sums are stored through to memory and are there before its ticket
        // is taken; whoever takes a tile's last one adds them in the parts' order.
        // (Release and acquire atomics would write back an XCD's whole L2.)
        __shared__ uint32_t s_last;
        uint64_t* slot = reinterpret_cast<uint64_t*>(
            a.slots + ((uint64_t)number * a.parts + part) * (B * B)) + threadIdx.x;
#pragma unroll
        for (int x = 0; x < TM; ++x)
#pragma unroll
            for (int y = 0; y < TN; ++y)
#pragma unroll
                for (int i = 0; i < 16; i += 2)
                    __hip_atomic_store(slot + ((x * TN + y) * 8 + i / 2) * THREADS,
                                       (uint64_t)__float_as_uint(g.acc[x][y][i + 1]) << 32 |
                                           __float_as_uint(g.acc[x][y][i]),
                                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __asm__ __volatile__("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0) {
            const uint32_t before = __hip_atomic_fetch_add(a.tickets + number, 1u, __ATOMIC_RELAXED,
                                                           __HIP_MEMORY_SCOPE_AGENT);
            s_last = before == a.parts - 1;
            if (s_last)
                __hip_atomic_store(a.tickets + number, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (!s_last)
            return;
        slot -= (uint64_t)part * (B * B / 2);
#pragma unroll
        for (int x = 0; x < TM; ++x)
#pragma unroll
            for (int y = 0; y < TN; ++y) {
                f32x16 sum;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    sum[i] = 0.0f;
                for (uint32_t o = 0; o < a.parts; ++o)
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const uint64_t two = __hip_atomic_load(
                            slot + (uint64_t)o * (B * B / 2) + ((x * TN + y) * 8 + i / 2) * THREADS,
                            __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                        sum[i] += __uint_as_float((uint32_t)two);
                        sum[i + 1] += __uint_as_float((uint32_t)(two >> 32));
                    }
                g.acc[x][y] = sum;
            }
    }

    // lane l holds column l % 32, rows 8 (r / 4) + 4 (l / 32) + r % 4 of a 32 x 32
    // product: four consecutive values of a row of C^T, and, after four lanes
    // exchanged theirs, of a row of C
    const uint32_t mp = padded(a.m), np = padded(a.n);
    float s_acc = a.s_acc, s_add = a.s_add, s_out = 1.0f;
    if (down || a.ends) {
        const OrthoLift& l = a.lift;
        const int now = above(down - l.now), next = above(down - l.next), b = above(2 * now - l.b);
        const int out = a.last ? halved_end(a.ends + next - now) : 0;
        s_acc = ldexpf(s_acc, l.acc[0] * now + l.acc[1] * next + l.acc[2] * b + a.ends - out);
        s_add = ldexpf(s_add, l.add[0] * now + l.add[1] * next + l.add[2] * b + a.ends - out);
        s_out = ldexpf(1.0f, out);
    }
    const _Float16* dt = a.dt ? a.dt + own : nullptr;
    _Float16 *c = a.c + own, *ct = a.ct + own;
    each_of<TM * TN>([&](auto number) {
        constexpr int x = number.value / TN, y = number.value % TN;
            const uint32_t j = j0 + wj + y * 32 + lane % 32;
            const uint32_t jq = j & ~3u;
            __asm__ __volatile__("" ::: "memory");  // not all of them at once: registers
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                const uint32_t i = i0 + wi + x * 32 + 8 * r4 + 4 * (lane / 32), iq = i + lane % 4;
                const bool in = j < a.n && i < mp;
                f16x4 dh, dl;
                if (dt && in) {
                    const _Float16* e = dt + half_at(j, i, a.n);
                    dh = *reinterpret_cast<const f16x4*>(e);
                    dl = *reinterpret_cast<const f16x4*>(e + kPiece);
                }
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    v[r] = g.acc[x][y][4 * r4 + r] * s_acc;
                    if (dt)
                        v[r] = fmaf((float)dh[r] + (float)dl[r], s_add, v[r]);
                    v[r] += i + r == j ? a.diag : 0.0f;
                    v[r] = i + r < a.m && j < a.n ? v[r] * s_out : 0.0f;
                }
                uint32_t w[4];
                if (a.last) {
                    if (a.transposed) {
                        if (j < a.n && i < a.m)
                            store_out(to, a.bf16, j * a.out_stride + i, a.m - i, v);
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            w[r] = __float_as_uint(v[r]);
                        transpose4(w);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            v[r] = __uint_as_float(w[r]);
                        if (iq < a.m && jq < a.n)
                            store_out(to, a.bf16, iq * a.out_stride + jq, a.n - jq, v);
                    }
                    continue;
                }
                f16x4 hi, lo;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    _Float16 vh, vl;
                    split(v[r], &vh, &vl);
                    hi[r] = vh;
                    lo[r] = vl;
                    w[r] = (uint32_t)__builtin_bit_cast(uint16_t, vl) << 16 |
                           __builtin_bit_cast(uint16_t, vh);
                }
                if (in) {
                    _Float16* o = ct + half_at(j, i, a.n);
                    *reinterpret_cast<f16x4*>(o) = hi;
                    *reinterpret_cast<f16x4*>(o + kPiece) = lo;
                }
                if (a.symmetric && ti == tj)
                    continue;
                transpose4(w);
                if (iq < a.m && jq < np) {
                    _Float16* o = c + half_at(iq, jq, a.m);
                    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                    *reinterpret_cast<u32x2*>(o) = u32x2{(w[0] & 0xffffu) | w[1] << 16,
                                                         (w[2] & 0xffffu) | w[3] << 16};
                    *reinterpret_cast<u32x2*>(o + kPiece) = u32x2{w[0] >> 16 | (w[1] & 0xffff0000u),
                                                                  w[2] >> 16 | (w[3] & 0xffff0000u)};
                }
            }
    });
}

// ---- small matrices ------------------------------------------------------------

constexpr int kSmallThreads = 1024, kSmallWaves = kSmallThreads / 64;

// Place, in halves, of the hi half of (r, c) in a matrix of `rows` rows in LDS: its
// pieces one after the other, the 16-byte chunks of a row exchanged as Stage's.
__device__ inline uint32_t small_at(uint32_t r, uint32_t c, uint32_t rows, uint32_t low)
{
    return (c / kPiece * rows + r) * (2 * kPiece) + ((c % kPiece / 8 + 4 * low) ^ r / 2 % 8) * 8 + c % 8;
}

// One tile: rows i0 .. of p by rows j0 .. of q, k columns (a multiple of 32).  Two
// sums of products, of which one need not wait for the other.
__device__ inline f32x16 small_tile(const _Float16* p, uint32_t p_rows, uint32_t i0, const _Float16* q,
                                    uint32_t q_rows, uint32_t j0, uint32_t k, uint32_t lane)
{
    f32x16 acc, low;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        acc[i] = low[i] = 0.0f;
    const uint32_t i = i0 + lane % 32, j = j0 + lane % 32;
#pragma unroll 1
    for (uint32_t c0 = 0; c0 < k; c0 += 32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t c = c0 + 16 * h + lane / 32 * 8;
            const auto at = [&](const _Float16* s, uint32_t r, uint32_t rows, uint32_t lower) {
                return *reinterpret_cast<const f16x8*>(s + small_at(r, c, rows, lower));
            };
            const f16x8 ph = at(p, i, p_rows, 0), qh = at(q, j, q_rows, 0);
            const f16x8 pl = at(p, i, p_rows, 1), ql = at(q, j, q_rows, 1);
            acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph, qh, acc, 0, 0, 0);
            low = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl, qh, low, 0, 0, 0);
            low = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph, ql, low, 0, 0, 0);
        }
    }
#pragma unroll
    for (int r = 0; r < 16; ++r)
        acc[r] += low[r];
    return acc;
}

// Four consecutive values of a row, from column c on (a multiple of 4).
__device__ inline void small_store(_Float16* s, uint32_t r, uint32_t c, uint32_t rows, const float (&v)[4])
{
    f16x4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        _Float16 h, l;
        split(v[i], &h, &l);
        hi[i] = h;
        lo[i] = l;
    }
    *reinterpret_cast<f16x4*>(s + small_at(r, c, rows, 0)) = hi;
    *reinterpret_cast<f16x4*>(s + small_at(r, c, rows, 1)) = lo;
}

__device__ inline void small_load(const _Float16* s, uint32_t r, uint32_t c, uint32_t rows, float (&v)[4])
{
    const f16x4 hi = *reinterpret_cast<const f16x4*>(s + small_at(r, c, rows, 0));
    const f16x4 lo = *reinterpret_cast<const f16x4*>(s + small_at(r, c, rows, 1));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = (float)hi[i] + (float)lo[i];
}

// All steps of a matrix by one workgroup, 16 waves, a block of a product each: what
// a product makes stays in registers until all waves have read what it replaces.
// 160 x 96, five steps: 41 us, and 91 by a launch a product; 40 of them 43.  Bound by
// the way from one product to the next: a step of one block is 2.1 us, of 160 x 96's
// fifteen 6.6, 3 of them matrix instructions (the loads of LDS one round ahead: 42
// us; only A's and B's lower triangle: 40, but 64 x 64 23 for 21).
template <class E>
__global__ __launch_bounds__(kSmallThreads) void k_ortho_small(OrthoPointers in, OrthoPointers out,
                                                               OrthoSmallArgs a)
{
    __shared__ __attribute__((aligned(16))) _Float16 s_all[kOrthoSmallBytes / 2];
    __shared__ double s_f[kSmallWaves];
    const typename E::T* p = static_cast<const typename E::T*>(in.p[blockIdx.x]);
    void* to = const_cast<void*>(out.p[blockIdx.x]);
    const bool tall = a.rows > a.cols;
    const uint32_t m = tall ? a.cols : a.rows, n = tall ? a.rows : a.cols;
    const uint32_t mp = padded(m), np = padded(n);
    _Float16 *x = s_all, *xt = x + 2 * mp * np, *ab = xt + 2 * mp * np;
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;

    // the matrix, four columns of a row at a time, rows of four neighbouring threads
    // one below the other
    constexpr int kHeld = 4;
    const uint32_t rp = padded(a.rows), cp = padded(a.cols), held = rp * cp / 4;
    float v[kHeld][4];
    double sum = 0.0;
    each_of<kHeld>([&](auto g) {
        const uint32_t i = g.value * kSmallThreads + threadIdx.x;
        const uint32_t r = i / cp * 4 + i % 4, c = i % cp / 4 * 4;
#pragma unroll
        for (int z = 0; z < 4; ++z)
            v[g.value][z] = i < held && r < a.rows && c + z < a.cols ? E::widen(p[r * a.x_stride + c + z])
                                                                     : 0.0f;
    });
    each_of<kHeld>([&](auto g) {
#pragma unroll
        for (int z = 0; z < 4; ++z)
            sum = fma((double)v[g.value][z], (double)v[g.value][z], sum);
    });
    const double norm = sqrt(block_sum<kSmallWaves>(sum, s_f)), by = norm + (double)a.eps;
    const int down = __builtin_amdgcn_readfirstlane(down_of(norm / by));
    const double up = ldexp(a.up, down) / by;
    each_of<kHeld>([&](auto g) {
        const uint32_t i = g.value * kSmallThreads + threadIdx.x;
        const uint32_t r = i / cp * 4, c = i % cp / 4 * 4;
        uint32_t w[4];
        float (&u)[4] = v[g.value];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            u[z] = (float)((double)u[z] * up);
            w[z] = __float_as_uint(u[z]);
        }
        transpose4(w);
        if (i < held) {
            small_store(tall ? xt : x, r + i % 4, c, rp, u);
#pragma unroll
            for (int z = 0; z < 4; ++z)
                u[z] = __uint_as_float(w[z]);
            small_store(tall ? x : xt, c + i % 4, r, cp, u);
        }
    });
    __syncthreads();

    // this wave's block of A and B, and of X
    const uint32_t mt = mp / 32, nt = np / 32, ai = wave / mt * 32, aj = wave % mt * 32;
    const uint32_t xi = wave / nt * 32, xj = wave % nt * 32;
    const bool has_a = wave < mt * mt, has_x = wave < mt * nt;
    f32x16 acc;
    // f(g, i, j): four consecutive values of C^T's row j, from column i on, are acc[4 g ..]
    const auto values = [&](uint32_t i0, uint32_t j0, auto f) {
        each_of<4>([&](auto g) {
            f(g, i0 + 8 * g.value + 4 * (lane / 32), j0 + lane % 32);
        });
    };
    float s_out = 1.0f;
    for (int step = 0;; ++step) {
        auto k = a.step[step];
        if (down || a.ends) {  // as the products' factors
            const bool last = step + 1 == a.steps;
            const int now = above(down - a.lift[step]), next = above(down - a.lift[step + 1]);
            const int b = above(2 * now - a.lift_b[step]), ends = last ? a.ends : 0;
            const int out = last ? halved_end(ends + next - now) : 0;
            k.b_acc = ldexpf(k.b_acc, b - 4 * now);
            k.b_add = ldexpf(k.b_add, b - 2 * now);
            k.x_acc = ldexpf(k.x_acc, next - now - b + ends - out);
            k.x_add = ldexpf(k.x_add, next - now + ends - out);
            s_out = ldexpf(1.0f, out);
        }
        if (has_a) {  // A = X X^T; A is its own transpose
            acc = small_tile(x, mp, ai, x, mp, aj, np, lane);
            values(ai, aj, [&](auto g, uint32_t i, uint32_t j) {
                float u[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    u[r] = acc[4 * g.value + r] * k.a;
                small_store(ab, j, i, mp, u);
            });
        }
        __syncthreads();
        if (has_a) {
            acc = small_tile(ab, mp, ai, ab, mp, aj, mp, lane);
            values(ai, aj, [&](auto g, uint32_t i, uint32_t j) {
                float d[4];
                small_load(ab, j, i, mp, d);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[4 * g.value + r] = fmaf(d[r], k.b_add, acc[4 * g.value + r] * k.b_acc);
            });
        }
        __syncthreads();
        if (has_a)
            values(ai, aj, [&](auto g, uint32_t i, uint32_t j) {
                const float u[4] = {acc[4 * g.value], acc[4 * g.value + 1], acc[4 * g.value + 2],
                                    acc[4 * g.value + 3]};
                small_store(ab, j, i, mp, u);
            });
        __syncthreads();
        if (has_x) {
            acc = small_tile(ab, mp, xi, xt, np, xj, mp, lane);
            values(xi, xj, [&](auto g, uint32_t i, uint32_t j) {
                float d[4];
                small_load(xt, j, i, np, d);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[4 * g.value + r] = fmaf(d[r], k.x_add, acc[4 * g.value + r] * k.x_acc);
            });
        }
        if (step + 1 == a.steps)
            break;
        __syncthreads();
        if (has_x)
            values(xi, xj, [&](auto g, uint32_t i, uint32_t j) {
                float u[4];
                uint32_t w[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    u[r] = acc[4 * g.value + r];
                    w[r] = __float_as_uint(u[r]);
                }
                small_store(xt, j, i, np, u);
                transpose4(w);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    u[r] = __uint_as_float(w[r]);
                small_store(x, i + lane % 4, j & ~3u, mp, u);
            });
        __syncthreads();
    }
    if (has_x)
        values(xi, xj, [&](auto g, uint32_t i, uint32_t j) {
            float u[4];
            uint32_t w[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                u[r] = acc[4 * g.value + r] * s_out;
                w[r] = __float_as_uint(u[r]);
            }
            if (tall) {
                if (j < n && i < m)
                    store_out(to, a.bf16, j * a.out_stride + i, m - i, u);
                return;
            }
            transpose4(w);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                u[r] = __uint_as_float(w[r]);
            const uint32_t iq = i + lane % 4, jq = j & ~3u;
            if (iq < m && jq < n)
                store_out(to, a.bf16, iq * a.out_stride + jq, n - jq, u);
        });
}

}  // namespace

hipError_t launch_ortho_small(const OrthoPointers& x, const OrthoPointers& out, int count,
                              const OrthoSmallArgs& a, hipStream_t s)
{
    if (a.bf16)
        hipLaunchKernelGGL(k_ortho_small<Elem<AR_BF16>>, dim3(count), dim3(kSmallThreads), 0, s, x, out, a);
    else
        hipLaunchKernelGGL(k_ortho_small<Elem<AR_FLOAT32>>, dim3(count), dim3(kSmallThreads), 0, s, x, out,
                           a);
    return hipGetLastError();
}

hipError_t launch_ortho_split(const OrthoPointers& x, int count, const OrthoSplitArgs& args, hipStream_t s)
{
    OrthoSplitArgs a = args;
    // a workgroup for every 8 vectors a thread
    a.nparts = (uint32_t)std::max<uint64_t>(
        1, std::min<uint64_t>(kNormParts, (uint64_t)a.rows * a.cols / (kThreads * (a.bf16 ? 64 : 32))));
    const dim3 parts(a.nparts, count);
    const dim3 tiles((padded(a.cols) + kTile - 1) / kTile, (padded(a.rows) + kTile - 1) / kTile, count);
    if (a.bf16) {
        hipLaunchKernelGGL(k_ortho_norm<Elem<AR_BF16>>, parts, dim3(kThreads), 0, s, x, a);
        hipLaunchKernelGGL(k_ortho_split<Elem<AR_BF16>>, tiles, dim3(kThreads), 0, s, x, a);
    } else {
        hipLaunchKernelGGL(k_ortho_norm<Elem<AR_FLOAT32>>, parts, dim3(kThreads), 0, s, x, a);
        hipLaunchKernelGGL(k_ortho_split<Elem<AR_FLOAT32>>, tiles, dim3(kThreads), 0, s, x, a);
    }
    return hipGetLastError();
}

namespace {

// What a tile's side costs, in microseconds: a piece of the tiles of one round
// of workgroups (`slots` of them are resident), when they are few and when the
// chip is full of them, and what a round takes besides (the first copies and
// the tile's way out; counted once a launch, twelve 1024 x 1024, five steps: 1.20
// ms, by rounds 1.16).  Measured at 64 x 64 to 4096 x 8192.  The wide tiles read
// LDS and the L2s less for a product and fill the chip's matrix cores (256 x 256:
// 4096 x 8192 with K = 4096 in 641 us, 1.29 PFLOP/s, what the library's float16
// product reaches; 128 x 128: 718), the small ones are spread over more of it
// (1024 x 1024: 64 x 64 15 us, 128 x 128 31, 256 x 256 86; the triangle of 4096 x
// 4096, K = 8192: 192 x 192, one round of 253 workgroups, 372 us, 128 x 128 503,
// 256 x 256, 136 workgroups, 428).
struct Form {
    uint32_t side, slots;
    double few, full, besides;
};
constexpr Form kForms[] = {{64, 512, 0.175, 0.48, 6.0},
                           {128, 256, 0.43, 0.75, 13.0},  // three stages
                           {128, 512, 0.59, 1.4, 13.0},   // two, and two workgroups on a CU
                           {192, 256, 0.75, 1.35, 25.0},
                           {256, 256, 1.17, 2.4, 35.0}};

double time_of(const Form& f, const OrthoProductArgs& a, int count)
{
    const uint64_t m = (a.m + f.side - 1) / f.side, n = (a.n + f.side - 1) / f.side;
    const uint64_t tiles = (uint64_t)count * (a.symmetric ? m * (m + 1) / 2 : m * n);
    const uint64_t rest = tiles % f.slots;
    double piece = (double)(tiles / f.slots) * f.full;
    if (rest)
        piece += f.few + (f.full - f.few) * (double)rest / f.slots;
    // a round's beginnings and ends, of which two workgroups of a CU hide half
    const double rounds = (double)((tiles + f.slots - 1) / f.slots);
    return piece * a.k + f.besides * (f.slots > 256 ? (rounds + 1.0) / 2.0 : rounds);
}

template <int B, int WM, int WN, int S, bool PARTS>
hipError_t launch_tiles(const OrthoPointers& out, int count, OrthoProductArgs a, hipStream_t s)
{
    a.tiles_m = (a.m + B - 1) / B;
    a.tiles_n = (a.n + B - 1) / B;
    a.tiles = a.symmetric ? a.tiles_m * (a.tiles_m + 1) / 2 : a.tiles_m * a.tiles_n;
    hipLaunchKernelGGL((k_ortho_product<B, WM, WN, S, PARTS>),
                       dim3(a.tiles * (uint32_t)count * (PARTS ? a.parts : 1)),
                       dim3(64 * (B / WM) * (B / WN)), 0, s, out, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ortho_product(const OrthoPointers& out, int count, const OrthoProductArgs& args,
                                hipStream_t s)
{
    OrthoProductArgs a = args;
    const Form* best = kForms;
    for (const Form& f : kForms)
        if (time_of(f, a, count) < time_of(*best, a, count))
            best = &f;
    switch (best - kForms) {
    case 1: return launch_tiles<128, 64, 64, 3, false>(out, count, a, s);
    case 2: return launch_tiles<128, 64, 64, 2, false>(out, count, a, s);
    case 3: return launch_tiles<192, 96, 96, 2, false>(out, count, a, s);
    case 4: return launch_tiles<256, 128, 64, 2, false>(out, count, a, s);
    }
    // a long way to go for few workgroups: its pieces are shared out (512 x 2048,
    // K = 2048, 36 tiles: 18.8 us whole, 13.8 by two parts)
    const uint64_t m = (a.m + 63) / 64, n = (a.n + 63) / 64;
    const uint64_t tiles = (uint64_t)count * (a.symmetric ? m * (m + 1) / 2 : m * n);
    a.parts = (uint32_t)std::min<uint64_t>(std::min<uint64_t>(kOrthoSlots / tiles, a.k / kOrthoPartPieces), kOrthoParts);
    if (tiles <= kOrthoTickets && a.parts > 1)
        return launch_tiles<64, 32, 32, 4, true>(out, count, a, s);
    return launch_tiles<64, 32, 32, 4, false>(out, count, a, s);
}

}  // namespace ar
