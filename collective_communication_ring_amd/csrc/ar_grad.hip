// ar_grad.hip -- the global 2-norm of many tensors, and their scaling by it.
//
// A launch takes a table of spans in its kernel arguments.  The tiles of all
// its spans are numbered through; workgroup b takes tiles b, b + grid, ...,
// with the next tile's loads in flight while it works on one.
//
// Squares are added in float64: every square of a float32 or bfloat16 is exact
// there (48 bits or fewer) and inside its range, so the sum needs no scaling.
#include "ar_norm_common.h"

namespace ar {
namespace {

constexpr int kTileNV = kGradTileVecs / kBlock;  // a thread's vectors of a tile

struct Tile {
    uint32_t span;
    uint32_t first, end;  // the span's tiles
    uint64_t word;     // the span's
    uint64_t offset;   // bytes from the span's start
    uint32_t halves;   // 16-bit units
    u32x4 r[kTileNV];
};

// The span that holds tile t is the last whose first tile is <= t.  Each lane
// of the wave compares its own entries, in one round of loads; a search by
// halves would wait for one entry after the other.
template <class Table>
__device__ inline void find_tile(const Table& tab, uint32_t t, Tile* o)
{
    int n = 0;
#pragma unroll
    for (int k = 0; k < Table::kSpans; k += 64)
        n += __popcll(__ballot(tab.first[k + (threadIdx.x & 63u)] <= t));
    const uint32_t s = (uint32_t)__builtin_amdgcn_readfirstlane(n) - 1;
    o->span = s;
    o->word = tab.span[s];
    o->first = tab.first[s];
    o->end = s + 1 < (uint32_t)tab.n ? tab.first[s + 1] : tab.tiles;
}

// Where tile t of its span lies.
__device__ inline void place_tile(uint32_t t, Tile* o)
{
    o->offset = (uint64_t)(t - o->first) * (kGradTileVecs * 16u);
    o->halves = t + 1 == o->end ? ((uint32_t)(o->word >> 48) & 0x1fffu) + 1 : kGradTileHalves;
}

// All loads of a tile in flight together, the same for both types.  Non-
// temporal: a list larger than the caches is read from memory twice anyway
// (and one that fits the memory-side cache is served by it all the same).
__device__ inline void load_tile(Tile* o)
{
    using Half = Elem<AR_BF16>;
    const uint16_t* p = reinterpret_cast<const uint16_t*>((o->word & kSpanAddress) + o->offset);
    if (o->halves == kGradTileHalves) {
#pragma unroll
        for (int k = 0; k < kTileNV; ++k)
            o->r[k] = __builtin_nontemporal_load(
                reinterpret_cast<const AnyVec<uint16_t>::type*>(p) + (k * kBlock + threadIdx.x));
    } else if (o->halves >= Half::VEC) {
#pragma unroll
        for (int k = 0; k < kTileNV; ++k)
            o->r[k] = load_vec<Half>(p, (k * kBlock + threadIdx.x) * 8u, o->halves);
    } else {
        const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < kTileNV; ++k)
            o->r[k] = zero;
        if (threadIdx.x == 0)
            for (uint32_t i = 0; i < o->halves; ++i)
                o->r[0][i / 2] |= (uint32_t)p[i] << (16 * (i % 2));
    }
}

// Before a tile's vectors are used: a cut-short tile's last one is moved into
// place, and those past its end are zero.
__device__ inline void fit_tile(Tile* o)
{
    using Half = Elem<AR_BF16>;
    if (o->halves != kGradTileHalves && o->halves >= Half::VEC)
#pragma unroll
        for (int k = 0; k < kTileNV; ++k)
            fit<Half>(o->r[k], (k * kBlock + threadIdx.x) * 8u, o->halves);
}

// Calls work(tile) for each of this workgroup's tiles.
template <class Table, class Work>
__device__ inline void for_tiles(const Table& tab, Work work)
{
    uint32_t t = blockIdx.x;
    if (t >= tab.tiles)
        return;
    Tile cur;
    find_tile(tab, t, &cur);
    place_tile(t, &cur);
    load_tile(&cur);
    for (;;) {
        t += gridDim.x;
        if (t >= tab.tiles || t < gridDim.x)
            break;
        Tile next;
        next.span = cur.span;
        next.word = cur.word;
        next.first = cur.first;
        next.end = cur.end;
        if (t >= cur.end)
            find_tile(tab, t, &next);
        place_tile(t, &next);
        load_tile(&next);
        fit_tile(&cur);
        work(cur);
        cur = next;
    }
    fit_tile(&cur);
    work(cur);
}

template <class E>
__device__ inline void add_squares(const Tile& tile, double (&acc)[2])
{
#pragma unroll
    for (int k = 0; k < kTileNV; ++k) {
        float v[E::VEC];
        widen_slot<E, E::VEC>(tile.r[k], v);
#pragma unroll
        for (int i = 0; i < E::VEC; ++i)
            acc[i & 1] = fma((double)v[i], (double)v[i], acc[i & 1]);
    }
}

__device__ inline bool last_ticket(uint32_t* ticket, uint32_t of)
{
    return __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == of - 1;
}

__global__ __launch_bounds__(kBlock, 4) void k_grad_norm(SpanTable<kNormSpans> tab, double* slots,
                                                         uint32_t* tickets, int live, float* norm)
{
    constexpr int W = kBlock / 64;
    __shared__ double s_d[W];
    __shared__ uint32_t s_last;
    double part[2] = {0.0, 0.0};
    for_tiles(tab, [&](const Tile& tile) {
        if (tile.word & kSpanBf16)
            add_squares<Elem<AR_BF16>>(tile, part);
        else
            add_squares<Elem<AR_FLOAT32>>(tile, part);
    });
    double acc = part[0] + part[1];
    acc = block_sum<W>(acc, s_d);
    // A slot is stored through to memory, and is there before its workgroup's
    // ticket is taken (the wait); whoever takes the last ticket reads all slots
    // from there.  Release and acquire atomics would write back and drop the
    // XCD's whole L2 for each workgroup.
    if (threadIdx.x == 0) {
        if ((int)blockIdx.x < live)
            acc += slots[blockIdx.x];
        __hip_atomic_store(slots + blockIdx.x, acc, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = 0;
        if (norm) {
            __asm__ __volatile__("s_waitcnt vmcnt(0)" ::: "memory");
            const uint32_t group = blockIdx.x / kTicketGroup;
            const uint32_t groups = (gridDim.x + kTicketGroup - 1) / kTicketGroup;
            const uint32_t left = gridDim.x - group * kTicketGroup;
            uint32_t* mine = tickets + group * kTicketLine;
            uint32_t* top = tickets + kTicketTop * kTicketLine;
            if (last_ticket(mine, left < kTicketGroup ? left : kTicketGroup)) {
                __hip_atomic_store(mine, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                s_last = groups == 1 || last_ticket(top, groups);
                if (s_last && groups > 1)
                    __hip_atomic_store(top, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
    }
    __syncthreads();
    if (!s_last)
        return;
    const int n = live > (int)gridDim.x ? live : (int)gridDim.x;
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += kBlock)
        sum += __hip_atomic_load(slots + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sum = block_sum<W>(sum, s_d);
    if (threadIdx.x == 0)
        *norm = (float)sqrt(sum);
}

template <class E>
__device__ inline void store_scaled(const Tile& tile, uint64_t dst, float coef)
{
    uint16_t* p = reinterpret_cast<uint16_t*>(dst + tile.offset);
#pragma unroll
    for (int k = 0; k < kTileNV; ++k) {
        float v[E::VEC];
        widen_slot<E, E::VEC>(tile.r[k], v);
#pragma unroll
        for (int i = 0; i < E::VEC; ++i)
            v[i] *= coef;
        store_vec<Elem<AR_BF16>, true>(p, narrow_slot<E>(v), (k * kBlock + threadIdx.x) * 8u,
                                       tile.halves);
    }
}

__device__ inline uint64_t output_of(const SpanOutputs& out, const Tile& tile)
{
    return out.dst[tile.span];
}

__device__ inline uint64_t output_of(const SpanShifts& out, const Tile& tile)
{
    const uint32_t i = (uint32_t)(tile.word >> 61) & 3u;
    static_assert(kClipShifts == 4, "two bits of a span's word");
    return (tile.word & kSpanAddress) +
           (i == 0 ? out.by[0] : i == 1 ? out.by[1] : i == 2 ? out.by[2] : out.by[3]);
}

template <class Table, class Out>
__global__ __launch_bounds__(kBlock, 4) void k_grad_clip(Table tab, Out out, const float* norm,
                                                         float max_norm)
{
    const float nv = *norm;
    const float c = max_norm / (nv + 1e-6f);
    const float coef = nv != nv ? nv : c < 1.0f ? c : 1.0f;
    for_tiles(tab, [&](const Tile& tile) {
        const uint64_t dst = output_of(out, tile);
        if (coef == 1.0f && dst == (tile.word & kSpanAddress))
            return;  // in place, unchanged
        if (tile.word & kSpanBf16)
            store_scaled<Elem<AR_BF16>>(tile, dst, coef);
        else
            store_scaled<Elem<AR_FLOAT32>>(tile, dst, coef);
    });
}

}  // namespace

hipError_t launch_grad_norm(const SpanTable<kNormSpans>& t, void* scratch, int live, int grid, float* norm,
                            hipStream_t s)
{
    double* slots = static_cast<double*>(scratch);
    hipLaunchKernelGGL(k_grad_norm, dim3(grid), dim3(kBlock), 0, s, t, slots,
                       reinterpret_cast<uint32_t*>(slots + kGradMaxBlocks), live, norm);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const SpanTable<kClipSpans>& t, const SpanOutputs& o, const float* norm,
                            float max_norm, int grid, hipStream_t s)
{
    hipLaunchKernelGGL((k_grad_clip<SpanTable<kClipSpans>, SpanOutputs>), dim3(grid), dim3(kBlock), 0,
                       s, t, o, norm, max_norm);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const SpanTable<kNormSpans>& t, const SpanShifts& o, const float* norm,
                            float max_norm, int grid, hipStream_t s)
{
    hipLaunchKernelGGL((k_grad_clip<SpanTable<kNormSpans>, SpanShifts>), dim3(grid), dim3(kBlock), 0, s,
                       t, o, norm, max_norm);
    return hipGetLastError();
}

}  // namespace ar
