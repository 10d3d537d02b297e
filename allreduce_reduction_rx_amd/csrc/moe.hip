// moe.hip -- tokens to the experts' rows and back (gfx950): the sort by
// expert with its gather, the weighted combination, and its gradient. The
// operations are defined in rx.h.
//
// All three move rows: their time is the rows' bytes over the memory rate at
// prefill sizes and the latency of one dependent chain of loads at decode
// sizes.
//
// The sort. The sorted place of pair i is a count: the pairs with a smaller
// expert, and the pairs before i with the same one, so the places are stable
// and do not depend on timing. For few pairs each token's
// workgroup counts for its own topk pairs over all ids (compares and adds
// over ids that sit in L2) in the one launch that gathers. Above, a launch
// places the pairs of a segment in each workgroup and another only moves
// rows; above kSelfCount one before them counts experts per segment.
#include "block_common.hpp"

namespace rx {
namespace {

constexpr int kGroup = 8;          // a token's pairs handled together
constexpr int kPlace = 1024;       // pairs placed at a time, threads of the kernels that count and place
constexpr size_t kSelfCount = 16384;
constexpr int kSegments = 128;     // at most: the placing kernel reads all segments' counts (12.9 us with 256 of 128 experts)

__device__ __forceinline__ int local_expert(int id, int first, int experts)
{
    const uint32_t e = (uint32_t)id - (uint32_t)first;   // ids below `first` wrap to large values
    return e < (uint32_t)experts ? (int)e : experts;     // `experts`: dropped
}

// Sums of c[0 .. N) over the workgroup: sum j in lane j of every wave.
template <int N>
__device__ __forceinline__ uint32_t block_counts(const uint32_t* c, uint32_t* lds)
{
    const int lane = lane_id(), wave = threadIdx.x / kWave, nw = blockDim.x / kWave;
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const uint32_t sum = wave_sum_u(c[j]);
        mine = lane == j ? sum : mine;
    }
    if (nw == 1)
        return mine;
    __syncthreads();   // the previous use of lds is over
    if (lane < N)
        lds[wave * N + lane] = mine;
    __syncthreads();
    mine = 0;
    if (lane < N)
        for (int w = 0; w < nw; ++w)
            mine += lds[w * N + lane];
    return mine;
}

// Segment s, expert e: pairs of the segment that go to e, in
// counts[s * experts + e].
__global__ __launch_bounds__(kPlace) void k_dispatch_count(DispatchArgs a)
{
    __shared__ uint32_t hist[kMaxExperts];
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x)
        hist[e] = 0;
    __syncthreads();
    const uint32_t lo = blockIdx.x * a.segment;
    const uint32_t hi = lo + a.segment < a.pairs ? lo + a.segment : a.pairs;
    for (uint32_t i = lo + threadIdx.x; i < hi; i += kPlace) {
        const int e = local_expert(a.ids[i], a.first, a.experts);
        if (e < a.experts)
            atomicAdd(&hist[e], 1u);   // integers: the order does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x)
        a.counts[(size_t)blockIdx.x * a.experts + e] = hist[e];
}

// The lanes whose key equals this lane's (keys of up to 11 bits).
__device__ __forceinline__ uint64_t same_key(int key, int bits)
{
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot(key >> b & 1);
        same &= key >> b & 1 ? set : ~set;
    }
    return same;
}

// Places the pairs of segment blockIdx.x; segment 0 writes the offsets too.
// SELF: every workgroup counts all ids itself instead of reading the
// segments' counts: up to kSelfCount pairs that is shorter than a launch
// (whole calls: 6000 pairs 8.2 against 10.7 us, 8192 10.6 and 12.2, 16384 13.7 and
// 14.0, 32768 23.1 and 21.7).
template <bool SELF>
__global__ __launch_bounds__(kPlace) void k_dispatch_place(DispatchArgs a)
{
    constexpr int kWaves = kPlace / kWave;
    __shared__ uint32_t base[kMaxExperts];               // the next place of each expert
    __shared__ uint32_t part[2][kPlace];
    __shared__ uint16_t hist[kWaves][kMaxExperts];
    __shared__ uint32_t wsum[kWaves];
    const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave, experts = a.experts;

    const uint32_t lo = blockIdx.x * a.segment;
    const uint32_t hi = lo + a.segment < a.pairs ? lo + a.segment : a.pairs;
    int id = lo + tid < hi ? a.ids[lo + tid] : -1;   // on its way meanwhile
    for (int i = tid; i < kWaves * kMaxExperts / 2; i += kPlace)
        reinterpret_cast<uint32_t*>(&hist[0][0])[i] = 0;
    // each expert's total, and its pairs before this segment
    uint32_t total = 0, before = 0;
    if constexpr (SELF) {
        part[0][tid] = part[1][tid] = 0;
        __syncthreads();
#pragma unroll 4
        for (uint32_t i = tid; i < a.pairs; i += kPlace) {
            const int e = local_expert(a.ids[i], a.first, experts);
            if (e < experts)
                atomicAdd(&part[i < lo][e], 1u);   // integers: the order does not matter
        }
        __syncthreads();
        if (tid < experts) {
            before = part[1][tid];
            total = part[0][tid] + before;
        }
    } else {
        // the segments' counts, dealt to the threads of an expert
        uint32_t width = kWave;
        while ((int)width < experts)
            width *= 2;
        const uint32_t e = tid % width, g = tid / width, groups = kPlace / width;
        if ((int)e < experts)
#pragma unroll 16
            for (uint32_t s = g; s < a.segments; s += groups) {
                const uint32_t c = a.counts[(size_t)s * experts + e];
                total += c;
                before += s < blockIdx.x ? c : 0;
            }
        part[0][tid] = total;
        part[1][tid] = before;
        __syncthreads();
        total = before = 0;
        if (g == 0)
            for (uint32_t i = 0; i < groups; ++i) {
                total += part[0][i * width + e];
                before += part[1][i * width + e];
            }
    }
    // the experts' starts: an exclusive sum over the workgroup
    const uint32_t incl = wave_incl(total);
    if (lane == kWave - 1)
        wsum[wave] = incl;
    __syncthreads();
    uint32_t start = incl - total, kept = 0;
    for (int w = 0; w < kWaves; ++w) {
        start += w < wave ? wsum[w] : 0;
        kept += wsum[w];
    }
    if (tid < experts) {
        base[tid] = start + before;
        if (blockIdx.x == 0)
            a.offsets[tid] = (int)start;
    }
    if (blockIdx.x == 0 && tid == 0)
        a.offsets[experts] = (int)kept;

    int bits = 1;
    while (1 << bits <= experts)   // keys 0 .. experts
        ++bits;
    for (uint32_t i0 = lo; i0 < hi; i0 += kPlace) {
        const uint32_t i = i0 + tid;
        if (i0 > lo)
            id = i < hi ? a.ids[i] : -1;
        const int key = i < hi ? local_expert(id, a.first, experts) : experts;
        const uint64_t same = same_key(key, bits);
        const uint32_t rank = __popcll(same & ((1ull << lane) - 1));
        const bool owned = key < experts, last = owned && (same >> lane) == 1;   // no higher lane has this key
        if (last)
            hist[wave][key] = (uint16_t)(rank + 1);
        __syncthreads();
        uint32_t p = 0;
        if (owned) {
            p = base[key] + rank;
            for (int w = 0; w < wave; ++w)
                p += hist[w][key];
            a.order[p] = (int)i;
        }
        if (i < hi)
            a.slots[i] = owned ? (int)p : -1;
        __syncthreads();   // base and hist have been read
        if (last) {
            atomicAdd(&base[key], rank + 1);
            hist[wave][key] = 0;
        }
        __syncthreads();
    }
    for (uint32_t p = (lo < kept ? kept : lo) + tid; p < hi; p += kPlace)
        a.order[p] = -1;
}

// Moves rows to the places in slots. OUT 1: copied; 2: quantized to INT8.
// Streaming stores, but not of rows that are no whole vectors: they share
// lines, which the caches then join (5003 x 6 x 2501 FP32: 88 -> 69 us).
template <int DT, int OUT, bool TAIL, int NV>
__global__ __launch_bounds__(256) void k_dispatch_rows(DispatchArgs a)
{
    constexpr int VE = Elem<DT>::kVE, EB = OUT == 1 ? Elem<DT>::kBytes : 1;
    __shared__ uint32_t lds[4];
    const int tid = threadIdx.x, bd = blockDim.x;
    const uint32_t t = blockIdx.x;
    const void* xrow = static_cast<const char*>(a.x) + (size_t)t * a.ld_x * Elem<DT>::kBytes;
    const int hidden = (int)a.hidden;
    const int nvec = (hidden + VE - 1) / VE;
    const int v0 = (int)(blockIdx.y * a.split_vecs);
    const int v1 = v0 + (int)a.split_vecs < nvec ? v0 + (int)a.split_vecs : nvec;
    u32x4 x[NV];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < NV; ++u)
            x[u] = ld_raw<DT, TAIL, OUT == 1>(xrow, base + u * bd, hidden);
#pragma unroll
        for (int u = 0; u < NV; ++u)
            x[u] = fixed<DT, TAIL>(x[u], base + u * bd, hidden);
    };
    load(v0 + tid);
    float scale = 1.0f, inv = 1.0f;
    if constexpr (OUT == 2) {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < NV; ++u)
            m = umax(m, vec_absmax<DT>(x[u]));
        // what the registers do not hold: the row's other splits, its rest
        for (int v = tid; v < nvec; v += bd)
            if (v < v0 || v >= v0 + NV * bd)
                m = umax(m, vec_absmax<DT>(ld_row<DT, TAIL>(xrow, v, hidden)));
        m = group_max<kWave>(m);
        if (bd > kWave) {
            if (lane_id() == 0)
                lds[tid / kWave] = m;
            __syncthreads();
            for (int w = 0; w < bd / kWave; ++w)
                m = umax(m, lds[w]);
        }
        i8_scale(bits_f32(m), scale, inv);
        if (blockIdx.y == 0)
            for (int j = tid; j < a.topk; j += bd) {
                const int s = a.slots[(size_t)t * a.topk + j];
                if (s >= 0)
                    a.row_scales[s] = scale;
            }
    }
    for (int base = v0 + tid; base - tid < v1; base += NV * bd) {
        if (base - tid > v0)
            load(base);
        uint32_t q[NV][2];
        if constexpr (OUT == 2)
#pragma unroll
            for (int u = 0; u < NV; ++u)
                i8_codes<DT>(x[u], inv, q[u]);
        for (int j = 0; j < a.topk; ++j) {
            const int s = a.slots[(size_t)t * a.topk + j];
            if (s < 0)
                continue;
            char* row = static_cast<char*>(a.rows) + (size_t)s * a.ld_rows * EB;
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int v = base + u * bd;
                if (v >= v1)
                    continue;
                if constexpr (OUT == 1)
                    st_row<DT, TAIL, !TAIL>(row, v, hidden, x[u]);
                else
                    st_codes<DT, TAIL>(row, v, hidden, q[u]);
            }
        }
    }
    // the rows that no pair owns, spread over the tokens' workgroups
    for (uint32_t p = (uint32_t)a.offsets[a.experts] + t; p < a.pairs; p += a.tokens) {
        char* row = static_cast<char*>(a.rows) + (size_t)p * a.ld_rows * EB;
        const u32x4 zero = {0, 0, 0, 0};
        const uint32_t none[2] = {0, 0};
        if (OUT == 2 && tid == 0 && blockIdx.y == 0)
            a.row_scales[p] = 1.0f;
        for (int v = v0 + tid; v < v1; v += bd) {
            if constexpr (OUT == 1)
                st_row<DT, TAIL, !TAIL>(row, v, hidden, zero);
            else
                st_codes<DT, TAIL>(row, v, hidden, none);
        }
    }
}

// Plan and rows in one launch. OUT 0: the plan alone; 1: rows copied; 2: rows
// quantized to INT8.
//
// A pair's place is the number of (expert, pair) keys below its own: one
// comparison and one addition of a carry for an id. The loop over the ids stays
// rolled: at these sizes a kernel's time is its way through code that no
// instruction cache holds yet (32 tokens x 8 choices x 8192 BF16 took 8.4 us with
// 16 ids at a time, unrolled, 6.2 rolled, and take 4.1 us in this form).
constexpr int kPairBits = 12;
static_assert(kDispatchCountAll <= 1 << kPairBits, "a key holds the pair's number");

__device__ __forceinline__ uint32_t pair_key(int expert, uint32_t pair) { return (uint32_t)expert << kPairBits | pair; }

// c[j] = the thread's ids whose keys are below to[j].
template <int N>
__device__ __forceinline__ void count_below(const DispatchArgs& a, const uint32_t* to, uint32_t* c)
{
#pragma unroll
    for (int j = 0; j < N; ++j)
        c[j] = 0;
#pragma unroll 1
    for (uint32_t i = threadIdx.x; i < a.pairs; i += blockDim.x) {
        const uint32_t key = pair_key(local_expert(a.ids[i], a.first, a.experts), i);
#pragma unroll
        for (int j = 0; j < N; ++j)
            c[j] += key < to[j];
    }
}

template <int DT, int OUT, bool TAIL>
__global__ __launch_bounds__(256) void k_dispatch(DispatchArgs a)
{
    __shared__ uint32_t lds[4 * (kGroup + 1)];
    __shared__ uint32_t tops[4];
    const int tid = threadIdx.x, bd = blockDim.x, lane = lane_id();
    const uint32_t t = blockIdx.x;

    if (t >= a.tokens) {
        // the offsets, kGroup experts a workgroup
        if (blockIdx.y)
            return;
        const int e0 = (int)(t - a.tokens) * kGroup;
        uint32_t c[kGroup], to[kGroup];
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
            to[j] = pair_key(e0 + j < a.experts ? e0 + j : a.experts, 0);
        count_below<kGroup>(a, to, c);
        const uint32_t n = block_counts<kGroup>(c, lds);
        if (tid < kGroup && e0 + tid <= a.experts)
            a.offsets[e0 + tid] = (int)n;
        return;
    }

    const void* xrow = static_cast<const char*>(a.x) + (size_t)t * a.ld_x * Elem<DT>::kBytes;
    constexpr int VE = Elem<DT>::kVE, XN = OUT == 2 ? 2 : 1;
    const int hidden = (int)a.hidden;
    const int nvec = (hidden + VE - 1) / VE;
    const int v0 = (int)(blockIdx.y * a.split_vecs);
    const int v1 = v0 + (int)a.split_vecs < nvec ? v0 + (int)a.split_vecs : nvec;
    u32x4 x[XN];
    if constexpr (OUT != 0)
#pragma unroll
        for (int u = 0; u < XN; ++u)
            x[u] = ld_raw<DT, TAIL>(xrow, v0 + tid + u * bd, hidden);

    float scale = 1.0f, inv = 1.0f;
    uint32_t kept = 0, top = 0;
    for (int j0 = 0; j0 < a.topk; j0 += kGroup) {
        const int nj = a.topk - j0 < kGroup ? a.topk - j0 : kGroup;
        const uint32_t i0 = t * (uint32_t)a.topk + (uint32_t)j0;
        // lane j of every wave: pair i0 + j
        const int key = lane < nj ? local_expert(a.ids[i0 + lane], a.first, a.experts) : a.experts;
        const bool here = key < a.experts;
        uint32_t c[kGroup + 1], to[kGroup + 1];
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
            to[j] = (uint32_t)__builtin_amdgcn_readlane((int)pair_key(key, i0 + lane), j);
        to[kGroup] = pair_key(a.experts, 0);   // all that are kept
        count_below<kGroup + 1>(a, to, c);
        if (OUT == 2 && j0 == 0) {
            uint32_t m = 0;
#pragma unroll
            for (int u = 0; u < XN; ++u)
                m = umax(m, vec_absmax<DT>(fixed<DT, TAIL>(x[u], v0 + tid + u * bd, hidden)));
            for (int v = tid; v < nvec; v += bd)   // the rest, and the other parts of a split row
                if (v < v0 || v >= v0 + XN * bd)
                    m = umax(m, vec_absmax<DT>(ld_row<DT, TAIL>(xrow, v, hidden)));
            top = group_max<kWave>(m);
            if (bd > kWave && lane == 0)
                tops[tid / kWave] = top;
        }
        const uint32_t place = block_counts<kGroup + 1>(c, lds);   // with several waves: barriers after tops is written
        kept = (uint32_t)__builtin_amdgcn_readlane((int)place, kGroup);
        if (OUT == 2 && j0 == 0) {
            if (bd > kWave)   // one wave has its row's largest already, and no barrier behind it
                for (int w = 0; w < bd / kWave; ++w)
                    top = umax(top, tops[w]);
            i8_scale(bits_f32(top), scale, inv);
        }
        if (tid < nj && blockIdx.y == 0) {
            a.slots[i0 + tid] = here ? (int)place : -1;
            if (here) {
                a.order[place] = (int)(i0 + tid);
                if constexpr (OUT == 2)
                    a.row_scales[place] = scale;
            }
        }
        if constexpr (OUT != 0) {
            const uint64_t mask = __ballot(here);
            auto emit = [&](int v, u32x4 xv) {
                uint32_t q[2];
                if constexpr (OUT == 2)
                    i8_codes<DT>(xv, inv, q);
                for (uint64_t left = mask; left; left &= left - 1) {
                    const size_t p = (uint32_t)__builtin_amdgcn_readlane((int)place, __builtin_ctzll(left));
                    if constexpr (OUT == 1)
                        st_row<DT, TAIL>(static_cast<char*>(a.rows) + p * a.ld_rows * Elem<DT>::kBytes, v, hidden, xv);
                    else
                        st_codes<DT, TAIL>(static_cast<char*>(a.rows) + p * a.ld_rows, v, hidden, q);
                }
            };
#pragma unroll
            for (int u = 0; u < XN; ++u)
                if (v0 + tid + u * bd < v1)
                    emit(v0 + tid + u * bd, fixed<DT, TAIL>(x[u], v0 + tid + u * bd, hidden));
            for (int v = v0 + tid + XN * bd; v < v1; v += bd)
                emit(v, ld_row<DT, TAIL>(xrow, v, hidden));
        }
    }

    // the rows that no pair owns, spread over the tokens' workgroups
    for (uint32_t p = kept + t; p < a.pairs; p += a.tokens) {
        if (tid == 0 && blockIdx.y == 0) {
            a.order[p] = -1;
            if constexpr (OUT == 2)
                a.row_scales[p] = 1.0f;
        }
        if constexpr (OUT == 1) {
            const u32x4 zero = {0, 0, 0, 0};
            for (int v = v0 + tid; v < v1; v += bd)
                st_row<DT, TAIL>(static_cast<char*>(a.rows) + (size_t)p * a.ld_rows * Elem<DT>::kBytes, v, hidden,
                                 zero);
        }
        if constexpr (OUT == 2) {
            const uint32_t zero[2] = {0, 0};
            for (int v = v0 + tid; v < v1; v += bd)
                st_codes<DT, TAIL>(static_cast<char*>(a.rows) + (size_t)p * a.ld_rows, v, hidden, zero);
        }
    }
}

// ---------------------------------------------------------------------------
// combine: a wave holds U x 64 vectors of one token's output
// ---------------------------------------------------------------------------

// Adds w_j rows[slot_j] for the N lowest set bits of `mask` (lane j holds
// slot j and weight j); all N rows' loads go out before the first addition.
template <int DT, bool TAIL, int U, int N>
__device__ __forceinline__ void combine_batch(const CombineArgs& a, uint64_t& mask, int slot, float w, int v, int hidden,
                                              float (*acc)[8])
{
    constexpr int VE = Elem<DT>::kVE;
    u32x4 x[N][U];
    float ws[N];
#pragma unroll
    for (int r = 0; r < N; ++r) {
        const int j = __builtin_ctzll(mask);
        mask &= mask - 1;
        const uint32_t s = (uint32_t)__builtin_amdgcn_readlane(slot, j);
        ws[r] = bits_f32((uint32_t)__builtin_amdgcn_readlane(__builtin_bit_cast(int, w), j));
        const char* row = static_cast<const char*>(a.rows) + (size_t)s * a.ld_rows * Elem<DT>::kBytes;
#pragma unroll
        for (int u = 0; u < U; ++u)
            x[r][u] = ld_raw<DT, TAIL, true>(row, v + u * kWave, hidden);
    }
#pragma unroll
    for (int r = 0; r < N; ++r)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[VE];
            unpack<DT>(fixed<DT, TAIL>(x[r][u], v + u * kWave, hidden), f);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                acc[u][k] += ws[r] * f[k];
        }
}

template <int DT, bool TAIL, int U>
__global__ __launch_bounds__(256) void k_combine(CombineArgs a)
{
    const int lane = lane_id();
    const size_t unit = (size_t)blockIdx.x * (blockDim.x / kWave) +
                        (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (unit >= a.tokens * a.chunks)
        return;
    const size_t t = unit / a.chunks;
    const int hidden = (int)a.hidden;
    const int v = (int)(unit - t * a.chunks) * U * kWave + lane;
    int slot = -1;
    float w = 1.0f;
    if (lane < a.topk) {
        slot = a.slots[t * a.topk + lane];
        if (a.weights)
            w = a.weights[t * a.topk + lane];
    }
    uint64_t mask = __ballot((uint32_t)slot < a.nrows);   // a negative slot is large as unsigned
    float acc[U][8] = {};
    while (mask) {
        switch (__builtin_popcountll(mask)) {
        case 1: combine_batch<DT, TAIL, U, 1>(a, mask, slot, w, v, hidden, acc); break;
        case 2: combine_batch<DT, TAIL, U, 2>(a, mask, slot, w, v, hidden, acc); break;
        case 3: combine_batch<DT, TAIL, U, 3>(a, mask, slot, w, v, hidden, acc); break;
        default: combine_batch<DT, TAIL, U, 4>(a, mask, slot, w, v, hidden, acc); break;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        st_row<DT, TAIL, true>(static_cast<char*>(a.out) + t * a.ld_out * Elem<DT>::kBytes, v + u * kWave, hidden,
                               pack<DT>(acc[u]));
}

// ---------------------------------------------------------------------------
// combine's gradient: a workgroup holds one token's d_out, NV vectors a
// thread at a time, and runs over the token's rows
// ---------------------------------------------------------------------------

template <int DT, bool TAIL, int NV, bool DW>
__global__ __launch_bounds__(256) void k_combine_backward(CombineBwdArgs a)
{
    constexpr int VE = Elem<DT>::kVE;
    __shared__ float part[4 * kGroup];
    const int tid = threadIdx.x, bd = blockDim.x, lane = lane_id(), wave = tid / kWave, nw = bd / kWave;
    const size_t t = blockIdx.x;
    const int hidden = (int)a.hidden;
    const int nvec = (hidden + VE - 1) / VE;
    const void* grow = static_cast<const char*>(a.d_out) + t * a.ld_d_out * Elem<DT>::kBytes;
    const int topk = t < a.tokens ? a.topk : 0;   // a call without tokens has workgroups for the rows' zeros
    for (int j0 = 0; j0 < topk; j0 += kGroup) {
        const int nj = topk - j0 < kGroup ? topk - j0 : kGroup;
        float dot[kGroup] = {};
        for (int base = tid; base < nvec; base += bd * NV) {
            float g[NV][VE];
#pragma unroll
            for (int u = 0; u < NV; ++u)
                unpack<DT>(ld_row<DT, TAIL>(grow, base + u * bd, hidden), g[u]);
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                const uint32_t s = j < nj ? (uint32_t)a.slots[t * a.topk + j0 + j] : ~0u;
                if (s >= a.nrows)
                    continue;
                const float w = a.weights ? a.weights[t * a.topk + j0 + j] : 1.0f;
                if constexpr (DW) {
                    const char* row = static_cast<const char*>(a.rows) + (size_t)s * a.ld_rows * Elem<DT>::kBytes;
                    u32x4 x[NV];
#pragma unroll
                    for (int u = 0; u < NV; ++u)
                        x[u] = ld_raw<DT, TAIL, true>(row, base + u * bd, hidden);
#pragma unroll
                    for (int u = 0; u < NV; ++u) {
                        float f[VE];
                        unpack<DT>(fixed<DT, TAIL>(x[u], base + u * bd, hidden), f);
#pragma unroll
                        for (int k = 0; k < VE; ++k)
                            dot[j] += g[u][k] * f[k];
                    }
                }
                char* drow = static_cast<char*>(a.d_rows) + (size_t)s * a.ld_d_rows * Elem<DT>::kBytes;
#pragma unroll
                for (int u = 0; u < NV; ++u) {
                    float f[VE];
#pragma unroll
                    for (int k = 0; k < VE; ++k)
                        f[k] = w * g[u][k];
                    st_row<DT, TAIL, !TAIL>(drow, base + u * bd, hidden, pack<DT>(f));
                }
            }
        }
        if constexpr (DW) {
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                dot[j] = wave_sum(dot[j]);
            __syncthreads();
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    part[wave * kGroup + j] = dot[j];
            __syncthreads();
            if (tid < nj) {
                float sum = 0.0f;   // a dropped pair's sum has no terms
                for (int w = 0; w < nw; ++w)
                    sum += part[w * kGroup + tid];
                a.d_weights[t * a.topk + j0 + tid] = sum;
            }
        }
    }
    const u32x4 zero = {0, 0, 0, 0};
    const int kept = *a.kept < 0 ? 0 : *a.kept;
    for (size_t p = (size_t)kept + t; p < a.nrows; p += gridDim.x)
        for (int v = tid; v < nvec; v += bd)
            st_row<DT, TAIL, true>(static_cast<char*>(a.d_rows) + p * a.ld_d_rows * Elem<DT>::kBytes, v, hidden, zero);
}

template <int OUT>
const void* dispatch_fn(int dtype, bool tail)
{
    if (dtype == 0)
        return tail ? (const void*)k_dispatch<0, OUT, true> : (const void*)k_dispatch<0, OUT, false>;
    return tail ? (const void*)k_dispatch<1, OUT, true> : (const void*)k_dispatch<1, OUT, false>;
}

template <int OUT, int NV>
const void* rows_fn(int dtype, bool tail)
{
    if (dtype == 0)
        return tail ? (const void*)k_dispatch_rows<0, OUT, true, NV> : (const void*)k_dispatch_rows<0, OUT, false, NV>;
    return tail ? (const void*)k_dispatch_rows<1, OUT, true, NV> : (const void*)k_dispatch_rows<1, OUT, false, NV>;
}

template <int U>
const void* combine_fn(int dtype, bool tail)
{
    if (dtype == 0)
        return tail ? (const void*)k_combine<0, true, U> : (const void*)k_combine<0, false, U>;
    return tail ? (const void*)k_combine<1, true, U> : (const void*)k_combine<1, false, U>;
}

template <int NV, bool DW>
const void* backward_fn(int dtype, bool tail)
{
    if (dtype == 0)
        return tail ? (const void*)k_combine_backward<0, true, NV, DW> : (const void*)k_combine_backward<0, false, NV, DW>;
    return tail ? (const void*)k_combine_backward<1, true, NV, DW> : (const void*)k_combine_backward<1, false, NV, DW>;
}

}  // namespace

uint32_t dispatch_segment(size_t pairs)
{
    const size_t per = (pairs + kSegments - 1) / kSegments;
    return (uint32_t)(per <= kPlace ? kPlace : (per + kPlace - 1) / kPlace * kPlace);
}

hipError_t launch_dispatch(const DispatchArgs& in, int dtype, int out, hipStream_t s)
{
    DispatchArgs a = in;
    void* params[] = {&a};
    // One launch counts every pair for every token, two place them first. Whole
    // calls, one launch against two: 32 tokens x 8 choices 4.6 and 7.2 us, 256 x 8 7.2 and
    // 9.1, 512 x 8 12.6 and 11.4, 4096 x 1 20.0 and 8.2.
    const bool seg = a.pairs > kDispatchCountAll || (size_t)a.tokens * a.pairs > (size_t)1 << 20;
    if (seg) {
        hipError_t e = hipSuccess;
        const bool self = a.pairs <= kSelfCount;
        if (!self)
            e = launch_logged("k_dispatch_count", (const void*)k_dispatch_count, dim3(a.segments), dim3(kPlace), params, s);
        if (e == hipSuccess)
            e = launch_logged("k_dispatch_place", self ? (const void*)k_dispatch_place<true> : (const void*)k_dispatch_place<false>,
                              dim3(a.segments), dim3(kPlace), params, s);
        if (e != hipSuccess || !out)
            return e;
    }
    const size_t nvec = out ? vectors(a.hidden, dtype) : 0;
    unsigned wg = threads_for(nvec, 256);
    if (!seg)   // threads for the ids too
        wg = threads_for(a.pairs, 256) > wg ? threads_for(a.pairs, 256) : wg;
    // enough workgroups to reach every CU when there are few tokens: rows
    // split into parts of at least one vector a thread
    size_t splits = 1;
    if (out && a.tokens) {
        const size_t want = 2 * (size_t)device_cu_count() / a.tokens;
        const size_t most = (nvec + wg - 1) / wg;
        splits = want < 1 ? 1 : want < most ? want : most;
        if (splits < 1)
            splits = 1;
    }
    a.split_vecs = (uint32_t)((nvec + splits - 1) / splits);
    const bool tail = out && partial(a.hidden, dtype);
    if (seg) {
        const size_t nv = (a.split_vecs + wg - 1) / wg;
        const void* fn = out == 1 ? nv <= 1 ? rows_fn<1, 1>(dtype, tail) : rows_fn<1, 2>(dtype, tail)
                         : nv <= 1 ? rows_fn<2, 1>(dtype, tail)
                         : nv <= 2 ? rows_fn<2, 2>(dtype, tail)
                                   : rows_fn<2, 4>(dtype, tail);
        return launch_logged("k_dispatch_rows", fn, dim3(a.tokens, (unsigned)splits), dim3(wg), params, s);
    }
    const void* fn = out == 0 ? dispatch_fn<0>(dtype, tail) : out == 1 ? dispatch_fn<1>(dtype, tail) : dispatch_fn<2>(dtype, tail);
    const unsigned offset_wgs = (unsigned)(a.experts / kGroup + 1);   // experts + 1 offsets
    return launch_logged("k_dispatch", fn, dim3(a.tokens + offset_wgs, (unsigned)splits), dim3(wg), params, s);
}

hipError_t launch_combine(const CombineArgs& in, int dtype, hipStream_t s)
{
    CombineArgs a = in;
    void* params[] = {&a};
    const size_t nvec = vectors(a.hidden, dtype);
    // two vectors a lane and four waves a workgroup for large calls (16384 tokens x 2
    // rows x 1024 BF16: 16.7 against 17.6 us), single waves for small ones (256 x 8 x 4096:
    // 4.6 against 5.0 us)
    const bool wide = a.tokens * nvec >= (size_t)device_cu_count() * 4096;
    const int u = wide ? 2 : 1;
    a.chunks = (nvec + (size_t)u * kWave - 1) / ((size_t)u * kWave);
    const size_t units = a.tokens * a.chunks;
    const unsigned wg = wide ? 256u : 64u;
    const size_t grid = (units * kWave + wg - 1) / wg;
    const void* fn = wide ? combine_fn<2>(dtype, partial(a.hidden, dtype)) : combine_fn<1>(dtype, partial(a.hidden, dtype));
    return launch_logged("k_combine", fn, dim3((unsigned)grid), dim3(wg), params, s);
}

hipError_t launch_combine_backward(const CombineBwdArgs& in, int dtype, hipStream_t s)
{
    CombineBwdArgs a = in;
    void* params[] = {&a};
    const size_t nvec = vectors(a.hidden, dtype);
    const bool tail = partial(a.hidden, dtype);
    const unsigned wg = threads_for(nvec, 256);
    const bool two = nvec > wg;
    const void* fn;
    if (a.d_weights)
        fn = two ? backward_fn<2, true>(dtype, tail) : backward_fn<1, true>(dtype, tail);
    else
        fn = two ? backward_fn<2, false>(dtype, tail) : backward_fn<1, false>(dtype, tail);
    const size_t clearing = (size_t)device_cu_count() * 8 < a.nrows ? (size_t)device_cu_count() * 8 : a.nrows;
    return launch_logged("k_combine_backward", fn, dim3((unsigned)(a.tokens ? a.tokens : clearing)), dim3(wg), params, s);
}

}  // namespace rx
