// gemm_fp4.hpp -- the kernels of the product of activations with 4-bit weights,
// dense or grouped by expert (gfx950). Defined in rx.h. Each type and group
// size is a translation unit of its own (gemm_fp4_*.hip).
#pragma once

#include "expert_tiles.hpp"

namespace rx {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// The eight weights of a dword, exactly.
__device__ __forceinline__ bf16x8 weights8(uint32_t w)
{
    struct {
        bf16x2 p[4];
    } x;
    x.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0);
    x.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1);
    x.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2);
    x.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3);
    return __builtin_bit_cast(bf16x8, x);
}

// Dword q of lane 16 i + r to dword i of lane 16 q + r: a lane loads 32
// neighbouring weights, and then holds 8 of each of the four 32s that its
// fifteen neighbours of the same column loaded.
__device__ __forceinline__ u32x4 turned(u32x4 x)
{
    auto a = __builtin_amdgcn_permlane32_swap(x[0], x[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(x[1], x[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{c[0], c[1], d[0], d[1]};
}

// Eight elements of a row from k0 on, k0 a multiple of 8; TAIL: zeros from k on.
template <int DT> struct Raw8 { u32x4 v[DT == 0 ? 2 : 1]; };

template <int DT, bool TAIL>
__device__ __forceinline__ Raw8<DT> ld_raw8(const void* row, int k0, int k)
{
    Raw8<DT> r;
    constexpr int N = DT == 0 ? 2 : 1;
#pragma unroll
    for (int i = 0; i < N; ++i)
        r.v[i] = TAIL ? ld_row<DT, true>(row, k0 / (8 / N) + i, k)
                      : ld16_any(static_cast<const char*>(row) + (uint32_t)(k0 * Elem<DT>::kBytes + i * 16));
    return r;
}

// One BF16 operand, or three that add up to the FP32 one: each the upper 16 bits
// of what the ones before leave.
template <int DT> struct Parts8 { bf16x8 p[DT == 0 ? 3 : 1]; };

template <int DT>
__device__ __forceinline__ Parts8<DT> parts8(const Raw8<DT>& r)
{
    Parts8<DT> x;
    if constexpr (DT == 1) {
        x.p[0] = __builtin_bit_cast(bf16x8, r.v[0]);
    } else {
        u32x4 w[3];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t a = r.v[j / 2][2 * (j & 1)], b = r.v[j / 2][2 * (j & 1) + 1];
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                w[n][j] = __builtin_amdgcn_perm(b, a, 0x07060302);   // the upper halves
                a = __builtin_bit_cast(uint32_t, bits_f32(a) - bits_f32(a & 0xFFFF0000u));
                b = __builtin_bit_cast(uint32_t, bits_f32(b) - bits_f32(b & 0xFFFF0000u));
            }
        }
#pragma unroll
        for (int n = 0; n < 3; ++n)
            x.p[n] = __builtin_bit_cast(bf16x8, w[n]);
    }
    return x;
}

// Chunk `c` of 128 weights of a row of b and their scales. Lane 16 q + r has 32
// neighbouring weights of row r; past the row the first ones, met by zeros of a.
template <int GR> struct Coded {
    u32x4 codes;
    float scale[128 / GR];
};

template <int GR>
__device__ __forceinline__ Coded<GR> ld_coded(const uint8_t* brow, const float* srow, uint32_t c, uint32_t kbytes, uint32_t groups)
{
    constexpr uint32_t SG = 128 / GR;
    Coded<GR> x;
    const uint32_t byte = c * 64 + (uint32_t)(lane_id() / 16) * 16, g = c * SG;
    x.codes = *reinterpret_cast<const u32x4*>(brow + (byte < kbytes ? byte : 0));
    if (g + SG <= groups) {
        if constexpr (SG == 4) {
            unpack<0>(ld16_any(srow + g), x.scale);
        } else {
#pragma unroll
            for (uint32_t i = 0; i < SG; ++i)
                x.scale[i] = srow[g + i];
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < SG; ++i)
            x.scale[i] = srow[g + i < groups ? g + i : groups - 1];
    }
    return x;
}

// Four results of a lane: rows m .. m + 3 of channel n.
template <int DT>
__device__ __forceinline__ void put4(const GemmFp4Args& a, const TileRows& rows, uint32_t m, uint32_t n, f32x4 v)
{
    if (n >= a.n)
        return;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (m + e < rows.hi) {
            char* p = static_cast<char*>(a.out) + ((size_t)(m + e) * a.ld_out + n) * Elem<DT>::kBytes;
            if constexpr (DT == 0)
                *reinterpret_cast<float*>(p) = v[e];
            else
                *reinterpret_cast<uint16_t*>(p) = (uint16_t)pack_bf16(v[e], 0.0f);
        }
}

// acc += the products of TM row fragments with the chunk's weights, group by
// group: exact products into a sum of the group's own, which the scale then
// joins to acc. A row's scaling waits until the next row's products are on their
// way. frag(r, m): the parts of row fragment r for the 32 of k number m.
template <int DT, int GR, int TM, int TN, class F>
__device__ __forceinline__ void multiply_chunk(const Coded<GR>* w, const F& frag, f32x4 (*acc)[TN])
{
    constexpr int SG = 128 / GR, MG = 4 / SG;
    u32x4 c[TN];
#pragma unroll
    for (int t = 0; t < TN; ++t)
        c[t] = turned(w[t].codes);
#pragma unroll
    for (int g = 0; g < SG; ++g) {
        bf16x8 b[MG][TN];
#pragma unroll
        for (int m = 0; m < MG; ++m)
#pragma unroll
            for (int t = 0; t < TN; ++t)
                b[m][t] = weights8(c[t][g * MG + m]);
        f32x4 sum[2][TN];
        auto scale = [&](int r) {
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[r][t][e] = __builtin_fmaf(sum[r & 1][t][e], w[t].scale[g], acc[r][t][e]);
        };
#pragma unroll
        for (int r = 0; r < TM; ++r) {
#pragma unroll
            for (int t = 0; t < TN; ++t)
                sum[r & 1][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < MG; ++m) {
                const Parts8<DT> x = frag(r, g * MG + m);
#pragma unroll
                for (int p = DT == 0 ? 2 : 0; p >= 0; --p)
#pragma unroll
                    for (int t = 0; t < TN; ++t)
                        sum[r & 1][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.p[p], b[m][t], sum[r & 1][t], 0, 0, 0);
            }
            if (r > 0)
                scale(r - 1);
            if (TM * TN >= 8)
                __builtin_amdgcn_sched_barrier(0);   // more at once would not fit the registers
        }
        scale(TM - 1);
    }
}

// Few rows: 16 TT rows x 16 NS channels a workgroup of KS x NS waves, KC of k a
// stage. Weights and scales go from memory to LDS without registers, each row's in one
// piece, NBUF - 1 stages ahead; so do the rows of a where they are BF16 and whole
// 16-byte units (WHOLE; TR of them), others go through registers one stage ahead, FP32
// as its three parts, so that each element is taken apart once. A wave has 16
// channels and every KS-th part of a stage; the KS sums meet in LDS in their order.
//
// Why by way of LDS: a load of 64 lanes that takes 64 bytes from each of 16 rows
// costs the cache 16 lines, as much as 2 KiB in one piece.
//
// Places in LDS: unit u (16 bytes) of row r sits where the sixteen rows of a read
// lie in different banks; the load picks its unit to match. Rows that are not
// there are not loaded, or are the last one again: their results are not used.
template <int DT, int GR, int TT, int TR, int KS, int NS, int KC, int NBUF, bool WHOLE>
__global__ __launch_bounds__(KS * NS * kWave) void k_gemm_fp4_stream(GemmFp4Args a)
{
    constexpr int EB = Elem<DT>::kBytes, BM = 16 * TT, BN = 16 * NS, kThreads = KS * NS * kWave;
    constexpr int P = DT == 0 ? 3 : 1, UX = KC / 8, UW = KC / 32, SG = 128 / GR, SR = KC / GR;   // units of a row, scales a chunk and a row
    constexpr int KW = KC / KS, kSteps = KW / 128;
    constexpr int SU = SR % 4 == 0 && BN * SR % 256 == 0 ? 4 : 1;                                    // scales of a load
    constexpr int kX = TR * UX, kW = BN * UW, kS = BN * SR;                        // units, units, scales of a stage
    constexpr int NX = (kX + kThreads - 1) / kThreads, NW = (kW + kThreads - 1) / kThreads;
    constexpr int NSC = (kS / SU + kThreads - 1) / kThreads, NS1 = (kS + kThreads - 1) / kThreads;
    constexpr int N = (WHOLE ? NX : 0) + NW + NSC;
    static_assert(KW % 128 == 0 && kX % kWave == 0 && kW % kWave == 0 && kS / SU % kWave == 0 && (NBUF == 2 || NBUF == 3), "");
    static_assert((kX % kThreads == 0 || kX < kThreads) && (kW % kThreads == 0 || kW < kThreads) && (kS / SU % kThreads == 0 || kS / SU < kThreads), "");
    struct Stage {
        u32x4 x[P][BM * UX];
        u32x4 w[kW];
        float s[kS];
    };
    __shared__ __align__(16) Stage ring[NBUF];
    static_assert(sizeof(ring) >= sizeof(f32x4) * KS * NS * TT * kWave && sizeof(ring) <= 160 * 1024, "");
    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int ks = wave % KS, ns = wave / KS, col = lane % 16, q = lane / 16;
    const Tiles tiles = count_tiles(a, BM);
    uint32_t tm, tn;
    if (!pick_tile(tiles, (a.n + BN - 1) / BN, tm, tn))
        return;
    const uint32_t n0 = tn * BN;
    const TileRows rows = find_tile(a, tiles, tm, BM);
    if (rows.lo >= rows.hi)
        return;
    if (rows.expert < 0) {
        zero_tile<DT>(a, rows, n0, BN);
        return;
    }
    const int k = (int)a.k, stages = (k + KC - 1) / KC;
    const uint32_t xunits = (uint32_t)k / 8, wunits = (uint32_t)(k + 31) / 32;
    const char* xbase = static_cast<const char*>(a.a) + (size_t)rows.lo * a.ld_a * EB;
    const uint8_t* wbase = a.b + (size_t)rows.expert * a.stride_b + (size_t)n0 * a.ld_b;
    const float* sbase = a.b_scales + ((size_t)rows.expert * a.n + n0) * a.groups;
    const uint32_t last_row = rows.hi - 1 - rows.lo, last_col = a.n - 1 - n0;
    auto wplace = [](int r, int u) { return u ^ (UW == 4 ? (r >> 2) & 3 : UW == 8 ? (r >> 1) & 7 : r & 15); };
    // scales of a row in units of SU
    auto splace = [](int r, int g) { return g ^ (r % 16 * SR / 64) / SU * SU; };
    // what this thread loads: below 2^32, 64 rows of a stride below 2^23 elements
    uint32_t xfrom[NX], xunit[NX], wfrom[NW], wunit[NW];
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        const int e = (i * kThreads + tid) % kX, r = e / UX;
        xfrom[i] = ((uint32_t)r < last_row ? (uint32_t)r : last_row) * (uint32_t)a.ld_a * EB;
        xunit[i] = (uint32_t)(e % UX ^ (r & 15));
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const int e = (i * kThreads + tid) % kW, r = e / UW;
        wfrom[i] = ((uint32_t)r < last_col ? (uint32_t)r : last_col) * (uint32_t)a.ld_b;
        wunit[i] = (uint32_t)wplace(r, e % UW);
    }
    // past k: the row's first unit, which nothing reads or zeros meet
    auto load = [&](int st, int buf) {
        Stage& to = ring[buf];
        if constexpr (WHOLE)
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const uint32_t u = (uint32_t)st * UX + xunit[i];
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(xbase + (xfrom[i] + (u < xunits ? u : 0) * 16)),
                                                 (__attribute__((address_space(3))) void*)&to.x[0][(i * kThreads + wave * kWave) % kX], 16, 0, 0);
            }
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const uint32_t u = (uint32_t)st * UW + wunit[i];
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(wbase + (wfrom[i] + (u < wunits ? u : 0) * 16)),
                                             (__attribute__((address_space(3))) void*)&to.w[(i * kThreads + wave * kWave) % kW], 16, 0, 0);
        }
        // scales: four at a time, one at a time where the row ends in the stage
        auto load_s = [&](auto count, auto each) {
            constexpr int U = each();
#pragma unroll
            for (int i = 0; i < count(); ++i) {
                const int e = (i * kThreads + tid) % (kS / U), r = e * U / SR;
                const uint32_t g = (uint32_t)(st * SR + splace(r, e * U % SR)), row = (uint32_t)r < last_col ? (uint32_t)r : last_col;
                auto from = (const __attribute__((address_space(1))) void*)(sbase + (row * a.groups + (g < a.groups ? g : 0)));
                auto at = (__attribute__((address_space(3))) void*)&to.s[(i * kThreads + wave * kWave) % (kS / U) * U];
                if constexpr (U == 4)
                    __builtin_amdgcn_global_load_lds(from, at, 16, 0, 0);
                else
                    __builtin_amdgcn_global_load_lds(from, at, 4, 0, 0);
            }
        };
        using std::integral_constant;
        if (SU > 1 && (uint32_t)(st + 1) * SR <= a.groups)
            load_s(integral_constant<int, NSC>(), integral_constant<int, SU>());
        else
            load_s(integral_constant<int, NS1>(), integral_constant<int, 1>());
    };
    // ... through registers: one stage ahead, asked for before the stage's other loads,
    // so that the wait for those need not count them
    constexpr int NXR = (BM * UX + kThreads - 1) / kThreads;
    static_assert(WHOLE || ((UX >= kWave ? UX % kWave == 0 : kWave % UX == 0) && (BM * UX % kThreads == 0 || BM * UX < kThreads)), "");
    Raw8<DT> xreg[WHOLE ? 1 : NXR];
    auto load_x = [&](int st) {
#pragma unroll
        for (int i = 0; i < NXR; ++i) {
            const uint32_t e = (uint32_t)(i * kThreads + tid), r = e / UX;
            if (r <= last_row && r < BM) {
                const char* row = xbase + r * (uint32_t)a.ld_a * EB;
                const int at = st * KC + (int)(e % UX) * 8;
                xreg[WHOLE ? 0 : i] = (st + 1) * KC <= k ? ld_raw8<DT, false>(row, at, k) : ld_raw8<DT, true>(row, at, k);
            }
        }
    };
    auto store_x = [&](int buf) {
#pragma unroll
        for (int i = 0; i < NXR; ++i) {
            const uint32_t e = (uint32_t)(i * kThreads + tid), r = e / UX;
            if (r <= last_row && r < BM) {
                const Parts8<DT> x = parts8<DT>(xreg[WHOLE ? 0 : i]);
#pragma unroll
                for (int p = 0; p < P; ++p)
                    ring[buf].x[p][r * UX + (e % UX ^ (r & 15))] = __builtin_bit_cast(u32x4, x.p[p]);
            }
        }
    };
    f32x4 acc[TT][1] = {};
    // chunk j of this wave's part of a stage; PART: k ends in the stage
    auto multiply = [&](const Stage& st, int left, auto part) {
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            const int k0 = ks * KW + j * 128;
            if (part() && k0 >= left)
                break;
            const int r = ns * 16 + col;
            Coded<GR> w[1];
            w[0].codes = st.w[r * UW + wplace(r, k0 / 32 + q)];
#pragma unroll
            for (int g = 0; g < SG; ++g)
                w[0].scale[g] = st.s[r * SR + splace(r, k0 / GR + g)];
            multiply_chunk<DT, GR, TT, 1>(w, [&](int t, int m) {
                Parts8<DT> f;
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    u32x4 x = st.x[p][(t * 16 + col) * UX + ((k0 / 8 + m * 4 + q) ^ col)];
                    if (WHOLE && part()) {
                        const int in = left - (k0 + m * 32 + q * 8);   // elements before k's end: all or none
#pragma unroll
                        for (int d = 0; d < 4; ++d)
                            x[d] = in > 0 ? x[d] : 0;
                    }
                    f.p[p] = __builtin_bit_cast(bf16x8, x);
                }
                return f;
            }, acc);
        }
    };
    if (!WHOLE && stages > 0)
        load_x(0);
    order();
#pragma unroll
    for (int st = 0; st < NBUF - 1; ++st)
        if (st < stages)
            load(st, st);
    int buf = 0;
    for (int st = 0; st < stages; ++st) {
        if constexpr (!WHOLE)
            store_x(buf);
        if (NBUF > 2 && st + 1 < stages)
            wait_loads<(NBUF - 2) * N>();   // the next stage's, which are behind this one's
        else
            wait_loads<0>();
        wait_lds();
        order();
        __builtin_amdgcn_s_barrier();   // this stage is there, and the one before is read
        order();
        if (!WHOLE && st + 1 < stages)
            load_x(st + 1);
        order();
        if (st + NBUF - 1 < stages)
            load(st + NBUF - 1, buf == 0 ? NBUF - 1 : buf - 1);
        if ((st + 1) * KC <= k)
            multiply(ring[buf], KC, std::integral_constant<bool, false>());
        else
            multiply(ring[buf], k - st * KC, std::integral_constant<bool, true>());
        buf = buf + 1 == NBUF ? 0 : buf + 1;
    }
    auto put = [&](int t, int group, f32x4 v) {
        put4<DT>(a, rows, rows.lo + (uint32_t)(t * 16 + q * 4), n0 + (uint32_t)(group * 16 + col), v);
    };
    if constexpr (KS == 1) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
            put(t, ns, acc[t][0]);
    } else {
        f32x4* joined = reinterpret_cast<f32x4*>(&ring[0]);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < TT; ++t)
            joined[((ns * TT + t) * KS + ks) * kWave + lane] = acc[t][0];
        __syncthreads();
        for (int i = wave; i < NS * TT; i += KS * NS) {
            f32x4 v = joined[i * KS * kWave + lane];
#pragma unroll
            for (int s = 1; s < KS; ++s)
                v += joined[(i * KS + s) * kWave + lane];
            put(i % TT, i / TT, v);
        }
    }
}

// FP32 rows times few channels: 16 rows x 16 channels a workgroup, whose eight waves
// take every eighth chunk of 128 of k; the sums meet in LDS in their order. All
// from memory to registers, D chunks ahead, the rows before the weights: loads
// return in order, so a row's chunk that was asked for after the weights would
// wait for them. Half the start of k_gemm_fp4_stream (13 x 1000 x 2051: 6.7
// against 7.9 us), but 16 lines of the cache a load (16 x 8192 x 8192: 39 against 21).
template <int DT, int GR>
__global__ __launch_bounds__(8 * kWave) void k_gemm_fp4_few(GemmFp4Args a)
{
    constexpr int KS = 8, BM = 16, BN = 16, EB = Elem<DT>::kBytes, D = 3;
    __shared__ f32x4 joined[KS][kWave];
    const int tid = threadIdx.x, lane = lane_id(), ks = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int col = lane % 16, q = lane / 16;
    const Tiles tiles = count_tiles(a, BM);
    uint32_t tm, tn;
    if (!pick_tile(tiles, (a.n + BN - 1) / BN, tm, tn))
        return;
    const uint32_t n0 = tn * BN;
    const TileRows rows = find_tile(a, tiles, tm, BM);
    if (rows.lo >= rows.hi)
        return;
    if (rows.expert < 0) {
        zero_tile<DT>(a, rows, n0, BN);
        return;
    }
    const int k = (int)a.k, chunks = (k + 127) / 128, mine = chunks > ks ? (chunks - ks + KS - 1) / KS : 0;
    const uint32_t kbytes = (uint32_t)(k + 31) / 32 * 16;
    const uint32_t last_row = rows.hi - 1 - rows.lo, last_col = a.n - 1 - n0, c = (uint32_t)col;
    const uint32_t xrow = c < last_row ? c : last_row, brow = c < last_col ? c : last_col;
    const char* xat = static_cast<const char*>(a.a) + ((size_t)rows.lo + xrow) * a.ld_a * EB;
    const uint8_t* bat = a.b + (size_t)rows.expert * a.stride_b + (size_t)(n0 + brow) * a.ld_b;
    const float* sat = a.b_scales + ((size_t)rows.expert * a.n + n0 + brow) * a.groups;
    Coded<GR> w[D][1];
    Raw8<DT> xs[D][4];
    auto load = [&](int i, int d) {
        const int at = ks + i * KS, k0 = at * 128 + q * 8;
#pragma unroll
        for (int s = 0; s < 4; ++s)
            xs[d][s] = at * 128 + 128 <= k ? ld_raw8<DT, false>(xat, k0 + 32 * s, k) : ld_raw8<DT, true>(xat, k0 + 32 * s, k);
        w[d][0] = ld_coded<GR>(bat, sat, (uint32_t)at, kbytes, a.groups);
    };
    f32x4 acc[1][1] = {};
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (d < mine)
            load(d, d);
    for (int i = 0; i < mine; i += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (i + d >= mine)
                break;
            multiply_chunk<DT, GR, 1, 1>(w[d], [&](int, int m) { return parts8<DT>(xs[d][m]); }, acc);
            if (i + d + D < mine)
                load(i + d + D, d);
        }
    }
    joined[ks][lane] = acc[0][0];
    __syncthreads();
    if (ks == 0) {
        f32x4 v = joined[0][lane];
#pragma unroll
        for (int s = 1; s < KS; ++s)
            v += joined[s][lane];
        put4<DT>(a, rows, rows.lo + (uint32_t)(q * 4), n0 + c, v);
    }
}

// Many rows: BM x BN results a workgroup of WM x WN waves, TM x TN products of 16 x
// 16 each. The rows' chunk of 128 of k is in LDS (FP32 as its three parts), the
// next one on its way there; the weights go to registers, and to BF16 by every
// wave that needs them, while the matrix cores run. Unit u of 8 elements of
// row r sits at u ^ r % 16, so that the sixteen rows of a read lie in different
// banks. DIRECT: BF16 rows that start 16-byte aligned go to LDS without
// registers; others, and a chunk that k ends in, through them.
template <int DT, int GR, int TM, int TN, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(WM * WN * kWave, 2) void k_gemm_fp4_tile(GemmFp4Args a)
{
    constexpr int BM = 16 * TM * WM, BN = 16 * TN * WN, EB = Elem<DT>::kBytes, P = DT == 0 ? 3 : 1;
    constexpr int kThreads = WM * WN * kWave, kRowsAPass = kThreads / 16, NP = BM / kRowsAPass, NBUF = DT == 0 ? 1 : 2;
    static_assert(BM % kRowsAPass == 0 && kRowsAPass % 16 == 0, "");
    __shared__ u32x4 xs[NBUF][P][BM][16];
    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int col = lane % 16, q = lane / 16;
    const Tiles tiles = count_tiles(a, BM);
    uint32_t tm, tn;
    if (!pick_tile(tiles, (a.n + BN - 1) / BN, tm, tn))
        return;
    const uint32_t n0 = tn * BN;
    const TileRows rows = find_tile(a, tiles, tm, BM);
    if (rows.lo >= rows.hi)
        return;
    if (rows.expert < 0) {
        zero_tile<DT>(a, rows, n0, BN);
        return;
    }
    const int k = (int)a.k, chunks = (k + 127) / 128;
    const uint32_t kbytes = (uint32_t)(k + 31) / 32 * 16;
    const char* xbase = static_cast<const char*>(a.a) + (size_t)rows.lo * a.ld_a * EB;
    const uint8_t* bbase = a.b + (size_t)rows.expert * a.stride_b + (size_t)n0 * a.ld_b;
    const float* sbase = a.b_scales + ((size_t)rows.expert * a.n + n0) * a.groups;
    const int wm = wave / WN * TM * 16, wn = wave % WN * TN * 16;
    const int xr = tid / 16, xu = tid % 16;   // this thread's row and unit of a pass
    const uint32_t last_row = rows.hi - 1 - rows.lo, last_col = a.n - 1 - n0;
    auto row_at = [&](int i) {   // of pass i, in bytes below 2^32
        const uint32_t r = (uint32_t)(i * kRowsAPass + xr);
        return (r < last_row ? r : last_row) * (uint32_t)a.ld_a * EB;
    };
    uint32_t bfrom[TN], sfrom[TN];
#pragma unroll
    for (int i = 0; i < TN; ++i) {
        const uint32_t r = (uint32_t)(wn + i * 16 + col), at = r < last_col ? r : last_col;
        bfrom[i] = at * (uint32_t)a.ld_b;
        sfrom[i] = at * a.groups;
    }
    Coded<GR> w[2][TN];
    auto load_w = [&](int c, Coded<GR>* to) {
#pragma unroll
        for (int t = 0; t < TN; ++t)
            to[t] = ld_coded<GR>(bbase + bfrom[t], sbase + sfrom[t], (uint32_t)c, kbytes, a.groups);
    };
    auto store_x = [&](int buf, int i, const Raw8<DT>& x) {
        const Parts8<DT> p = parts8<DT>(x);
#pragma unroll
        for (int j = 0; j < P; ++j)
            xs[buf][j][i * kRowsAPass + xr][xu ^ (xr & 15)] = __builtin_bit_cast(u32x4, p.p[j]);
    };
    f32x4 acc[TM][TN] = {};
    int buf = 0;
    auto frag = [&](int r, int m) {
        Parts8<DT> f;
#pragma unroll
        for (int p = 0; p < P; ++p)
            f.p[p] = __builtin_bit_cast(bf16x8, xs[buf][p][wm + r * 16 + col][(m * 4 + q) ^ col]);
        return f;
    };
    if constexpr (DT == 1) {
        auto load_x = [&](int c, int to) {
            if (DIRECT && c * 128 + 128 <= k) {
                // LDS is written in lane order: the lane picks the unit that belongs there
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    __builtin_amdgcn_global_load_lds(
                        (const __attribute__((address_space(1))) void*)(xbase + (row_at(i) + (uint32_t)(c * 256 + (xu ^ (xr & 15)) * 16))),
                        (__attribute__((address_space(3))) void*)&xs[to][0][i * kRowsAPass + wave * 4][0], 16, 0, 0);
            } else {
#pragma unroll 1
                for (int i = 0; i < NP; i += 4) {
                    Raw8<DT> x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[j] = ld_raw8<DT, true>(xbase + row_at(i + j), c * 128 + xu * 8, k);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        store_x(to, i + j, x[j]);
                }
            }
        };
        static_assert(NP % 4 == 0, "");
        if (chunks > 0) {
            load_x(0, 0);
            load_w(0, w[0]);
        }
        for (int c = 0; c < chunks; c += 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (c + h >= chunks)
                    break;
                // this chunk has arrived, and every wave is done with the one before
                wait_loads<0>();
                wait_lds();
                order();
                __builtin_amdgcn_s_barrier();
                order();
                if (c + h + 1 < chunks) {
                    load_x(c + h + 1, h ^ 1);
                    load_w(c + h + 1, w[h ^ 1]);
                }
                buf = h;
                multiply_chunk<DT, GR, TM, TN>(w[h], frag, acc);
            }
        }
    } else {
        Raw8<DT> x[NP];
        auto load_x = [&](int c) {
            if (c * 128 + 128 <= k) {
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    x[i] = ld_raw8<DT, false>(xbase + row_at(i), c * 128 + xu * 8, k);
            } else {
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    x[i] = ld_raw8<DT, true>(xbase + row_at(i), c * 128 + xu * 8, k);
            }
        };
        if (chunks > 0) {
            load_x(0);
            load_w(0, w[0]);
        }
        for (int c = 0; c < chunks; c += 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (c + h >= chunks)
                    break;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    store_x(0, i, x[i]);
                __syncthreads();
                if (c + h + 1 < chunks) {
                    load_x(c + h + 1);
                    load_w(c + h + 1, w[h ^ 1]);
                }
                multiply_chunk<DT, GR, TM, TN>(w[h], frag, acc);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < TM; ++r)
#pragma unroll
        for (int t = 0; t < TN; ++t)
            put4<DT>(a, rows, rows.lo + (uint32_t)(wm + r * 16 + q * 4), n0 + (uint32_t)(wn + t * 16 + col), acc[r][t]);
}

// A call's workgroups: whole rounds of the XCDs for the tiles with an expert and
// for those without.
inline hipError_t launch_grid(GemmFp4Args& a, const void* fn, const char* name, size_t bm, size_t bn, unsigned threads, hipStream_t s)
{
    void* params[] = {&a};
    const size_t grid = (row_tiles(a, bm) * ((a.n + bn - 1) / bn) + 2 * kXcds) / kXcds * kXcds;
    return launch_logged(name, fn, dim3((unsigned)grid), dim3(threads), params, s);
}

template <int DT, int GR, int TT, int TR, int KS, int NS, int KC, int NBUF, bool WHOLE>
hipError_t launch_stream(GemmFp4Args& a, const char* name, hipStream_t s)
{
    return launch_grid(a, (const void*)k_gemm_fp4_stream<DT, GR, TT, TR, KS, NS, KC, NBUF, WHOLE>, name, 16 * TT,
                       16 * NS, KS * NS * kWave, s);
}

template <int DT, int GR, int TM, int TN, int WM, int WN, bool DIRECT>
hipError_t launch_tile(GemmFp4Args& a, hipStream_t s)
{
    return launch_grid(a, (const void*)k_gemm_fp4_tile<DT, GR, TM, TN, WM, WN, DIRECT>, "k_gemm_fp4_tile", 16 * TM * WM,
                       16 * TN * WN, WM * WN * kWave, s);
}

// A kind of workgroup: its tile, how many a CU takes, and the microseconds that
// 1024 of k take it alone on its CU, and with the CU full.
struct Kind {
    double bm, bn, per_cu, alone, full;
};

// Estimated time. The kinds' figures are measured at 8192 and 4096 of k, with
// groups of 128 (32: 5 to 15% more, alike for all). Up to one workgroup a CU runs at
// `alone`; a CU that fills up goes over to `full`. With experts the number of tiles is known
// to about half a tile each.
inline double estimate(const GemmFp4Args& a, const Kind& x)
{
    const double cus = device_cu_count();
    double tm = (double)((a.rows + (size_t)x.bm - 1) / (size_t)x.bm);
    if (a.offsets) {
        const double owners = (double)a.experts < a.rows ? (double)a.experts : a.rows;
        tm = a.rows / x.bm + 0.5 * owners;
        tm = tm < owners ? owners : tm;
    }
    const double tn = (double)((a.n + (size_t)x.bn - 1) / (size_t)x.bn), t = tm * tn / cus, k = a.k / 1024.0, start = 0.5;
    if (((double)row_tiles(a, (size_t)x.bm) * tn + 16.0) * 512.0 >= 4294967296.0)
        return 1e300;   // threads of one launch
    if (t <= 1.0)
        return start + k * x.alone;
    if (t <= x.per_cu)
        return start + k * (x.alone + (x.full - x.alone) * (t - 1.0) / (x.per_cu - 1.0));
    const double r = t / x.per_cu, up = (double)(long long)r + (r > (double)(long long)r ? 1.0 : 0.0);
    const double rounds = x.per_cu > 1.0 ? r + 0.25 < up ? r + 0.25 : up : a.offsets ? t + 0.5 : up;
    return rounds * (start + k * x.full);
}

// The kinds, and where another would go wrong (us, groups of 128):
//   BF16                          16x16 16x32 16x64 32x32 32x128 64x32 64x128 128x128
//   13 x 4096 x 8192                9.2  10.3
//   16 x 8192 x 8192               15.0  11.4  38.9
//   32 x 8192 x 8192                                 15.5  30.7
//   64 x 8192 x 8192                                              22.4   52
//   512 x 8192 x 8192                                              159   88    95
//   1024 x 8192 x 8192                                                  182   161
//   64 experts x 4 x 4096 x 4096          190   120
//   64 experts x 24 x 4096 x 4096                     270   163
//   64 experts x 48 x 4096 x 4096                                  415  240   340
//   FP32                            few  16x32 16x64        32x128       64x128
//   13 x 1000 x 2051                6.7   7.9
//   16 x 8192 x 8192                 39    21
//   512 x 8192 x 8192                                        246          214
//   64 experts x 4 x 4096 x 4096          296   180
//   64 experts x 48 x 4096 x 4096                            510          468
template <int DT, int GR>
hipError_t launch_fp4(const GemmFp4Args& in, hipStream_t s)
{
    GemmFp4Args a = in;
    constexpr Kind kBf16[] = {{16, 32, 1, 1.05, 1.05}, {16, 64, 4, 2.6, 7.5}, {32, 32, 1, 1.6, 1.6}, {32, 128, 2, 3.5, 9.5},
                              {64, 32, 1, 2.5, 2.5}, {64, 128, 2, 6.2, 10.6}, {128, 128, 2, 11.3, 19.7},
                              {16, 16, 1, 0.75, 0.75}};
    constexpr Kind kFp32[] = {{16, 32, 1, 2.2, 2.2}, {16, 64, 2, 4.3, 5.6}, {32, 128, 2, 8.1, 15.4}, {64, 128, 2, 20.0, 26.0},
                              {16, 16, 1, 2.0, 2.0}};
    const bool whole = DT == 1 && (uintptr_t)a.a % 16 == 0 && a.ld_a % 8 == 0 && a.k % 8 == 0;
    const Kind* kinds = DT == 0 ? kFp32 : kBf16;
    const int n = DT == 0 ? 5 : whole ? 8 : 7;
    int best = 0;
    double cost = 1e301;
    for (int i = 0; i < n; ++i) {
        const double c = estimate(a, kinds[i]);
        if (c < cost) {
            cost = c;
            best = i;
        }
    }
    if constexpr (DT == 0) {
        switch (best) {
        case 0: return launch_stream<0, GR, 1, 16, 4, 2, 512, 2, false>(a, "k_gemm_fp4_stream 16x32", s);
        case 1: return launch_stream<0, GR, 1, 16, 1, 4, 256, 2, false>(a, "k_gemm_fp4_stream 16x64", s);
        case 2: return launch_stream<0, GR, 2, 32, 1, 8, 128, 2, false>(a, "k_gemm_fp4_stream 32x128", s);
        case 3: return launch_tile<0, GR, 4, 2, 1, 4, false>(a, s);
        default: return launch_grid(a, (const void*)k_gemm_fp4_few<0, GR>, "k_gemm_fp4_few", 16, 16, 8 * kWave, s);
        }
    } else if (whole) {
        const bool four = a.rows <= 4;   // fewer rows to load: 1 x 8192 x 8192 9.9 against 11.2 us
        switch (best) {
        case 0: return four ? launch_stream<1, GR, 1, 4, 4, 2, 1024, 3, true>(a, "k_gemm_fp4_stream 16x32, four rows", s) : launch_stream<1, GR, 1, 16, 4, 2, 1024, 3, true>(a, "k_gemm_fp4_stream 16x32", s);
        case 1: return launch_stream<1, GR, 1, 16, 1, 4, 256, 2, true>(a, "k_gemm_fp4_stream 16x64", s);
        case 2: return launch_stream<1, GR, 2, 32, 4, 2, 512, 3, true>(a, "k_gemm_fp4_stream 32x32", s);
        case 3: return launch_stream<1, GR, 2, 32, 1, 8, 256, 2, true>(a, "k_gemm_fp4_stream 32x128", s);
        case 4: return launch_stream<1, GR, 4, 64, 4, 2, 512, 2, true>(a, "k_gemm_fp4_stream 64x32", s);
        case 5: return launch_stream<1, GR, 4, 64, 1, 8, 128, 3, true>(a, "k_gemm_fp4_stream 64x128", s);
        case 6: return launch_tile<1, GR, 4, 4, 2, 2, true>(a, s);
        default: return four ? launch_stream<1, GR, 1, 4, 8, 1, 1024, 2, true>(a, "k_gemm_fp4_stream 16x16, four rows", s) : launch_stream<1, GR, 1, 16, 8, 1, 1024, 2, true>(a, "k_gemm_fp4_stream 16x16", s);
        }
    } else {
        switch (best) {
        case 0: return launch_stream<1, GR, 1, 16, 4, 2, 1024, 3, false>(a, "k_gemm_fp4_stream 16x32, rows by way of registers", s);
        case 1: return launch_stream<1, GR, 1, 16, 1, 4, 256, 2, false>(a, "k_gemm_fp4_stream 16x64, rows by way of registers", s);
        case 2: return launch_stream<1, GR, 2, 32, 4, 2, 512, 3, false>(a, "k_gemm_fp4_stream 32x32, rows by way of registers", s);
        case 3: return launch_stream<1, GR, 2, 32, 1, 8, 256, 2, false>(a, "k_gemm_fp4_stream 32x128, rows by way of registers", s);
        case 4: return launch_stream<1, GR, 4, 64, 4, 2, 512, 2, false>(a, "k_gemm_fp4_stream 64x32, rows by way of registers", s);
        case 5: return launch_stream<1, GR, 4, 64, 1, 8, 128, 3, false>(a, "k_gemm_fp4_stream 64x128, rows by way of registers", s);
        default: return launch_tile<1, GR, 4, 4, 2, 2, false>(a, s);
        }
    }
}

}  // namespace
}  // namespace rx
