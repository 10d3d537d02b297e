// expert_tiles.hpp -- what the products share (gemm_i8.hip, gemm_fp4.hip): the
// tiles of a call, dense or with a matrix for each expert, and their order;
// results that fill no whole vector; waits for loads that go to LDS.
#pragma once

#include <utility>

#include "block_common.hpp"

namespace rx {
namespace {

// The rows of expert e, clamped to the matrix.
template <class A>
__device__ __forceinline__ void expert_rows(const A& a, int e, uint32_t& lo, uint32_t& hi)
{
    const int o0 = a.offsets[e], o1 = a.offsets[e + 1];
    lo = o0 < 0 ? 0 : (uint32_t)o0 < a.rows ? (uint32_t)o0 : a.rows;
    hi = o1 < 0 ? 0 : (uint32_t)o1 < a.rows ? (uint32_t)o1 : a.rows;
    hi = hi > lo ? hi : lo;
}

// The row tiles of a call: each expert's rows start a tile of their own;
// past the last, tiles of the rows that no expert owns. Every wave counts
// them for itself, 64 experts at a time, and keeps the first 64.
struct Tiles {
    uint32_t owned, end, total;   // tiles with an expert; the last expert's end; all tiles
    uint32_t lo, hi, incl;        // expert `lane`: its rows, the tiles up to its last
};

template <class A>
__device__ __forceinline__ uint32_t tiles_to(const A& a, int e, uint32_t bm, uint32_t& lo, uint32_t& hi)
{
    lo = hi = 0;
    if (e < a.experts)
        expert_rows(a, e, lo, hi);
    return wave_incl((hi - lo + bm - 1) / bm);
}

template <class A>
__device__ __forceinline__ Tiles count_tiles(const A& a, uint32_t bm)
{
    Tiles t = {};
    if (!a.offsets) {
        t.owned = t.total = (a.rows + bm - 1) / bm;
        t.end = a.rows;
        return t;
    }
    for (int e0 = 0; e0 < a.experts; e0 += kWave) {
        uint32_t lo, hi;
        const uint32_t incl = tiles_to(a, e0 + lane_id(), bm, lo, hi);
        if (e0 == 0) {
            t.lo = lo;
            t.hi = hi;
            t.incl = incl;
        }
        t.owned += (uint32_t)__builtin_amdgcn_readlane((int)incl, kWave - 1);
        t.end = (uint32_t)__builtin_amdgcn_readlane((int)hi, (a.experts - e0 < kWave ? a.experts - e0 : kWave) - 1);
    }
    t.total = t.owned + (a.rows - t.end + bm - 1) / bm;
    return t;
}

// The rows [lo, hi) of row tile `tm` and their expert, -1 past the last's.
struct TileRows {
    uint32_t lo, hi;
    int expert;
};

template <class A>
__device__ __forceinline__ TileRows find_tile(const A& a, const Tiles& t, uint32_t tm, uint32_t bm)
{
    if (!a.offsets) {
        const uint32_t lo = tm * bm;
        return {lo, lo + bm < a.rows ? lo + bm : a.rows, 0};
    }
    if (tm >= t.owned) {
        const uint32_t lo = t.end + (tm - t.owned) * bm;
        return {lo, lo + bm < a.rows ? lo + bm : a.rows, -1};
    }
    uint32_t base = 0, lo = t.lo, hi = t.hi, incl = t.incl;
    // offsets past the first 64 are read a second time: should another stream
    // write them meanwhile, the walk still ends, without a tile
    for (int e0 = 0; e0 < a.experts;) {
        const uint64_t past = __ballot(base + incl > tm);
        if (past) {
            const int l = __builtin_ctzll(past);
            const uint32_t own = (uint32_t)__builtin_amdgcn_readlane((int)incl, l) + base;   // tiles up to its last
            const uint32_t rlo = (uint32_t)__builtin_amdgcn_readlane((int)lo, l);
            const uint32_t rhi = (uint32_t)__builtin_amdgcn_readlane((int)hi, l);
            const uint32_t first = own - (rhi - rlo + bm - 1) / bm;
            const uint32_t at = rlo + (tm - first) * bm;
            return {at, at + bm < rhi ? at + bm : rhi, e0 + l};
        }
        base += (uint32_t)__builtin_amdgcn_readlane((int)incl, kWave - 1);
        e0 += kWave;
        incl = tiles_to(a, e0 + lane_id(), bm, lo, hi);
    }
    return {0, 0, 0};
}

constexpr uint32_t kTileGroup = 8;

// Workgroup -> tile. Workgroups go to the XCDs in turn, and each XCD has its
// own L2: an XCD takes a run of tiles of its own, eight row tiles by the
// columns, so that the 32 it works on together share rows and columns. The
// tiles without an expert come after, dealt to all XCDs alike.
__device__ __forceinline__ bool pick_tile(const Tiles& t, uint32_t ntn, uint32_t& tm, uint32_t& tn)
{
    const uint32_t owned = t.owned * ntn, per = (owned + kXcds - 1) / kXcds;
    const uint32_t i = blockIdx.x / kXcds, xcd = blockIdx.x % kXcds;
    if (i >= per) {
        const uint32_t tile = (i - per) * kXcds + xcd;
        tm = t.owned + tile / ntn;
        tn = tile % ntn;
        return tm < t.total;
    }
    const uint32_t tile = xcd * per + i;
    if (tile >= owned)
        return false;
    const uint32_t group = tile / (kTileGroup * ntn), in = tile % (kTileGroup * ntn), first = group * kTileGroup;
    const uint32_t size = t.owned - first < kTileGroup ? t.owned - first : kTileGroup;
    tm = first + in % size;
    tn = in / size;
    return true;
}

// Eight results of one row from column n on; `full`: all below a.n.
template <int DT, class A>
__device__ __forceinline__ void st_out8(const A& a, size_t m, uint32_t n, const float* v)
{
    char* p = static_cast<char*>(a.out) + (m * a.ld_out + n) * Elem<DT>::kBytes;
    if (n + 8 <= a.n) {
        st16_any(p, pack<DT>(v));
        if constexpr (DT == 0)
            st16_any(p + 16, pack<DT>(v + 4));
    } else {
        for (int e = 0; e < 8; ++e)
            if (n + e < a.n) {
                if constexpr (DT == 0)
                    reinterpret_cast<float*>(p)[e] = v[e];
                else
                    reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)pack_bf16(v[e], 0.0f);
            }
    }
}

template <int DT, class A>
__device__ void zero_tile(const A& a, const TileRows& r, uint32_t n0, uint32_t bn)
{
    const float zero[8] = {};
    const uint32_t per = bn / 8;
    for (uint32_t i = threadIdx.x; i < (r.hi - r.lo) * per; i += blockDim.x) {
        const uint32_t n = n0 + i % per * 8;
        if (n < a.n)
            st_out8<DT>(a, r.lo + i / per, n, zero);
    }
}

// s_waitcnt vmcnt(n) alone.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
}
// s_waitcnt lgkmcnt(0) alone.
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// f(0), f(1), ... with constant arguments.
template <class F, int... I>
__device__ __forceinline__ void unrolled_of(const F& f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void unrolled(const F& f)
{
    unrolled_of(f, std::make_integer_sequence<int, N>());
}

__device__ __forceinline__ void order() { asm volatile("" ::: "memory"); }

// Row tiles of a call, at most. Experts: each may end in a partial tile, and
// so may the rows past them.
template <class A>
size_t row_tiles(const A& a, size_t bm)
{
    const size_t owners = (size_t)a.experts < a.rows ? (size_t)a.experts : a.rows;
    return a.offsets ? a.rows / bm + owners + 1 : (a.rows + bm - 1) / bm;
}

}  // namespace
}  // namespace rx
