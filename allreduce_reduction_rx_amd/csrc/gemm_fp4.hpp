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
            x.scale[i] = g + i < groups ? srow[g + i] : 0.0f;
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
template <int DT, int GR, int TM, class F>
__device__ __forceinline__ void multiply_chunk(const Coded<GR>& w, const F& frag, f32x4 (&acc)[TM])
{
    constexpr int SG = 128 / GR, MG = 4 / SG;
    const u32x4 c = turned(w.codes);
#pragma unroll
    for (int g = 0; g < SG; ++g) {
        bf16x8 b[MG];
#pragma unroll
        for (int m = 0; m < MG; ++m)
            b[m] = weights8(c[g * MG + m]);
        f32x4 sum[2];
        auto scale = [&](int r) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[r][e] = __builtin_fmaf(sum[r & 1][e], w.scale[g], acc[r][e]);
        };
#pragma unroll
        for (int r = 0; r < TM; ++r) {
            sum[r & 1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < MG; ++m) {
                const Parts8<DT> x = frag(r, g * MG + m);
#pragma unroll
                for (int p = DT == 0 ? 2 : 0; p >= 0; --p)
                    sum[r & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.p[p], b[m], sum[r & 1], 0, 0, 0);
            }
            if (r > 0)
                scale(r - 1);
        }
        scale(TM - 1);
    }
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave); }

// What rows of a and scales are past k: weights may be anything there, and 0 times
// infinity is NaN.
__device__ const u32x4 kNothing = {0, 0, 0, 0};

// A stage of KC of k for BM rows of a and BN of b in LDS, and the loads that fill
// it: weights and scales from memory to LDS without registers, each row's in one
// piece; so do the rows of a where they are BF16 and whole 16-byte units (WHOLE; TR
// of them), others go through registers, FP32 as its three parts, so that each
// element is taken apart once.
//
// Why by way of LDS: a load of 64 lanes that takes 64 bytes from each of 16 rows
// keeps the cache busy for 35 cycles, one that takes 128 bytes and more for 20 (30 and 50
// bytes a cycle and CU), and 64 single words from as many lines for 65.
//
// Places in LDS: unit u (16 bytes) of row r sits where the sixteen rows of a read
// lie in different banks; the load picks its unit to match. Rows that are not
// there are not loaded, or are the last one again: their results are not used.
template <int DT, int GR, int BM, int BN, int TR, int KC, int T, bool WHOLE>
struct Stager {
    static constexpr int EB = Elem<DT>::kBytes, P = DT == 0 ? 3 : 1;
    static constexpr int UX = KC / 8, UW = KC / 32, SR = KC / GR;                 // units of a row, scales of a row
    static constexpr int SU = SR % 4 == 0 && BN * SR % 256 == 0 ? 4 : 1;          // scales of a load
    static constexpr int kX = TR * UX, kW = BN * UW, kS = BN * SR;                // units, units, scales of a stage
    static constexpr int NX = WHOLE ? (kX + T - 1) / T : 0, NW = (kW + T - 1) / T;
    static constexpr int NS = (kS / SU + T - 1) / T, NS1 = (kS + T - 1) / T;
    static constexpr int N = NX + NW + NS;                                        // a thread's loads, at least
    static constexpr int NXR = WHOLE ? 0 : (BM * UX + T - 1) / T;
    static_assert(kX % kWave == 0 && kW % kWave == 0 && kS / SU % kWave == 0, "");
    static_assert((kX % T == 0 || kX < T) && (kW % T == 0 || kW < T) && (kS / SU % T == 0 || kS / SU < T), "");
    static_assert(WHOLE || ((UX >= kWave ? UX % kWave == 0 : kWave % UX == 0) && (BM * UX % T == 0 || BM * UX < T)), "");
    static constexpr int RX = TR < 16 ? TR : BM;   // fewer than a fragment's: its other rows are these again
    struct Rows {
        u32x4 x[P][RX * UX];
    };
    struct Weights {
        u32x4 w[kW];
        float s[kS];
    };
    struct Stage : Rows, Weights {};

    const char* xbase;
    const uint8_t* wbase;
    const float* sbase;
    uint32_t last_row, last_col, ld_a, ld_b, groups, xunits, wunits;
    int k, wave;
    Raw8<DT> xreg[WHOLE ? 1 : NXR];

    __device__ __forceinline__ Stager(const GemmFp4Args& a, const TileRows& rows, uint32_t n0)
    {
        k = (int)a.k;
        wave = wave_id();
        xunits = (uint32_t)k / 8;
        wunits = (uint32_t)(k + 31) / 32;
        xbase = static_cast<const char*>(a.a) + (size_t)rows.lo * a.ld_a * EB;
        wbase = a.b + (size_t)rows.expert * a.stride_b + (size_t)n0 * a.ld_b;
        sbase = a.b_scales + ((size_t)rows.expert * a.n + n0) * a.groups;
        last_row = rows.hi - 1 - rows.lo;
        last_col = a.n - 1 - n0;
        ld_a = (uint32_t)a.ld_a * EB;   // below 2^25: 128 rows lie within 32 bits
        ld_b = (uint32_t)a.ld_b;
        groups = a.groups;
    }
    static __device__ __forceinline__ int wplace(int r, int u)
    {
        return u ^ (UW == 4 ? (r >> 2) & 3 : UW == 8 ? (r >> 1) & 7 : r & 15);
    }
    static __device__ __forceinline__ int splace(int r, int g) { return g ^ (r % 16 * SR / 64) / SU * SU; }
    static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) { return a < b ? a : b; }

    template <int B>
    static __device__ __forceinline__ void copy(const void* from, void* to)   // the builtin wants a literal size
    {
        if constexpr (B == 16)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                             (__attribute__((address_space(3))) void*)to, 16, 0, 0);
        else
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                             (__attribute__((address_space(3))) void*)to, 4, 0, 0);
    }
    template <int U>
    __device__ __forceinline__ void load_scales(int st, Weights& to, int i) const
    {
        const int e = (i * T + (int)threadIdx.x) % (kS / U), r = e * U / SR;
        const uint32_t g = (uint32_t)(st * SR + splace(r, e * U % SR));
        const float* from = sbase + (least((uint32_t)r, last_col) * groups + g);
        copy<4 * U>(g < groups ? from : (const float*)&kNothing, &to.s[(i * T + wave * kWave) % (kS / U) * U]);
    }
    // Load I of stage st. Weights past k: the row's first ones, which zeros meet.
    template <int I, class To>
    __device__ __forceinline__ void load(int st, To& to) const
    {
        const int tid = (int)threadIdx.x;
        if constexpr (I < NX) {
            const int e = (I * T + tid) % kX, r = e / UX;
            const uint32_t u = (uint32_t)(st * UX + (e % UX ^ (r & 15)));
            const char* from = xbase + (least((uint32_t)r, last_row) * ld_a + u * 16);
            copy<16>(u < xunits ? from : (const char*)&kNothing, &to.x[0][(I * T + wave * kWave) % kX]);
        } else if constexpr (I < NX + NW) {
            constexpr int i = I - NX;
            const int e = (i * T + tid) % kW, r = e / UW;
            const uint32_t u = (uint32_t)(st * UW + wplace(r, e % UW));
            copy<16>(wbase + (least((uint32_t)r, last_col) * ld_b + (u < wunits ? u : 0) * 16), &to.w[(i * T + wave * kWave) % kW]);
        } else if constexpr (I < N) {
            // four scales at a time, one at a time where the row ends in the stage
            constexpr int i = I - NX - NW;
            if (SU > 1 && (uint32_t)(st + 1) * SR <= groups) {
                load_scales<SU>(st, to, i);
            } else {
#pragma unroll
                for (int j = i * NS1 / NS; j < (i + 1) * NS1 / NS; ++j)
                    load_scales<1>(st, to, j);
            }
        }
    }
    // The rows that go through registers: a stage's loads, asked for before the
    // stage's other loads, so that the wait for those need not count them.
    template <int I>
    __device__ __forceinline__ void load_x(int st)
    {
        if constexpr (I < NXR) {
            const uint32_t e = (uint32_t)(I * T) + threadIdx.x, r = e / UX;
            if (r <= last_row && r < BM) {
                const char* row = xbase + r * ld_a;
                const int at = st * KC + (int)(e % UX) * 8;
                xreg[I] = (st + 1) * KC <= k ? ld_raw8<DT, false>(row, at, k) : ld_raw8<DT, true>(row, at, k);
            }
        }
    }
    __device__ __forceinline__ void store_x(Rows& to)
    {
        if constexpr (NXR > 0)
#pragma unroll
            for (int i = 0; i < NXR; ++i) {
                const uint32_t e = (uint32_t)(i * T) + threadIdx.x, r = e / UX;
                if (r <= last_row && r < BM) {
                    const Parts8<DT> x = parts8<DT>(xreg[i]);
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        to.x[p][r * UX + (e % UX ^ (r & 15))] = __builtin_bit_cast(u32x4, x.p[p]);
                }
            }
    }
    // Eight elements of row r (r % 16 = lane % 16) from k0 of the stage on.
    static __device__ __forceinline__ Parts8<DT> rows_of(const Rows& st, int r, int k0)
    {
        Parts8<DT> f;
        r = TR < 16 ? r % TR : r;
#pragma unroll
        for (int p = 0; p < P; ++p)
            f.p[p] = __builtin_bit_cast(bf16x8, st.x[p][r * UX + (k0 / 8 ^ (r & 15))]);
        return f;
    }
    // Dword q of unit m of weight row r.
    static __device__ __forceinline__ uint32_t codes_of(const Weights& st, int r, int m, int q)
    {
        return reinterpret_cast<const uint32_t*>(&st.w[r * UW + wplace(r, m)])[q];
    }
    static __device__ __forceinline__ float scale_of(const Weights& st, int r, int g) { return st.s[r * SR + splace(r, g)]; }
};

// Waits for a stage's loads and the waves: the stage is there, and the one
// before has been read. `next`: N loads of a later stage may still be on their way.
template <int N>
__device__ __forceinline__ void open_stage(bool next)
{
    if (N > 0 && next)
        wait_loads<N>();
    else
        wait_loads<0>();
    wait_lds();
    order();
    __builtin_amdgcn_s_barrier();
    order();
}

// Few rows: 16 TT rows x 16 NS channels a workgroup of KS x NS waves, KC of k a
// stage, DX - 1 stages of rows and DW - 1 of weights on their way. How many pays is
// measured: 64 x 8192 x 8192 in groups of 32 with weights from memory 34.5 us with one of each and 27.5
// with two of weights, 13 x 4096 x 8192 12.0 with one of each, 9.1 with two and three, but
// 256 rows of 64 experts, whose three or four workgroups a CU wait for each other less, 17.8
// with one and 21 with two. A wave has 16 channels and every KS-th part of a
// stage; the KS sums meet in LDS in their order. 1 x 8192 x 8192 takes 10.3 us with the weights'
// 36 MB from memory and 9.4 with them in the last-level cache, 32 rows 16.1 and 14.7 (their rows,
// which every workgroup reads again by way of L2, are less than half of that): bound by the start and
// the end, and by stages whose wait, LDS reads, conversions and products follow each
// other with two waves a SIMD (waves wait 61% and 47% of their cycles, matrix cores are busy 7% and 9%).
template <int DT, int GR, int TT, int TR, int KS, int NS, int KC, int DX, int DW, bool WHOLE>
__global__ __launch_bounds__(KS * NS * kWave) void k_gemm_fp4_stream(GemmFp4Args a)
{
    constexpr int BM = 16 * TT, BN = 16 * NS, SG = 128 / GR, KW = KC / KS;
    using S = Stager<DT, GR, BM, BN, TR, KC, KS * NS * kWave, WHOLE>;
    constexpr int NWS = S::N - S::NX;
    static_assert(KW % 128 == 0 && DX >= 2 && DW >= DX && (WHOLE || DX == DW), "");
    // as many of both: one ring, whose places take one offset (one ring 114 us for 32 x 8
    // rows of 64 experts, two 119)
    constexpr bool ONE = DX == DW;
    __shared__ __align__(16) typename S::Stage ring[DX];
    __shared__ __align__(16) typename S::Rows xring[DX];
    __shared__ __align__(16) typename S::Weights wring[DW];
    static_assert((ONE ? sizeof(ring) : sizeof(xring) + sizeof(wring)) <= 160 * 1024, "");
    static_assert(KS == 1 || sizeof(xring) >= sizeof(f32x4) * KS * NS * TT * kWave, "");
    auto rows_at = [&](int b) -> typename S::Rows& {
        if constexpr (ONE) return ring[b]; else return xring[b];
    };
    auto weights_at = [&](int b) -> typename S::Weights& {
        if constexpr (ONE) return ring[b]; else return wring[b];
    };
    const int lane = lane_id(), wave = wave_id(), ks = wave % KS, ns = wave / KS, col = lane % 16, q = lane / 16;
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
    S s(a, rows, n0);
    const int k = (int)a.k, stages = (k + KC - 1) / KC;
    f32x4 acc[TT] = {};
    // this wave's part of a stage
    auto multiply = [&](const typename S::Rows& xs, const typename S::Weights& ws, int left) {
#pragma unroll
        for (int j = 0; j < KW / 128; ++j) {
            const int k0 = ks * KW + j * 128;
            if (k0 >= left)
                break;
            const int r = ns * 16 + col;
            Coded<GR> w;
            w.codes = ws.w[r * S::UW + S::wplace(r, k0 / 32 + q)];
#pragma unroll
            for (int g = 0; g < SG; ++g)
                w.scale[g] = S::scale_of(ws, r, k0 / GR + g);
            multiply_chunk<DT, GR, TT>(w, [&](int t, int m) { return S::rows_of(xs, t * 16 + col, k0 + m * 32 + q * 8); }, acc);
        }
    };
    auto load_x = [&](int st) {
        unrolled<S::NXR>([&](auto i) { s.template load_x<i()>(st); });
        order();
    };
    auto load_rows = [&](int st, typename S::Rows& to) { unrolled<S::NX>([&](auto i) { s.template load<i()>(st, to); }); };
    auto load_weights = [&](int st, typename S::Weights& to) { unrolled<NWS>([&](auto i) { s.template load<S::NX + i()>(st, to); }); };
    if (S::NXR > 0 && stages > 0)
        load_x(0);
#pragma unroll
    for (int at = 1 - DW; at < 0; ++at) {   // as if the stages before had sent them
        if (at + DX > 0 && at + DX - 1 < stages)
            load_rows(at + DX - 1, rows_at((at + DX - 1) % DX));
        if (at + DW > 0 && at + DW - 1 < stages)
            load_weights(at + DW - 1, weights_at((at + DW - 1) % DW));
    }
    int bx = 0, bw = 0;
    for (int st = 0; st < stages; ++st) {
        s.store_x(rows_at(bx));
        // Loads return in their order: what went out after this stage's rows (which,
        // with DW > DX, went out after its weights) may still be on its way.
        if (ONE)
            open_stage<(DX - 2) * S::N>(st + DX - 2 < stages);
        else if (st + DW - 2 < stages)
            open_stage<(DX - 2) * S::N + NWS>(true);
        else
            open_stage<(DX - 2) * S::NX>(st + DX - 2 < stages);
        if (S::NXR > 0 && st + 1 < stages)
            load_x(st + 1);
        const int nx = bx == 0 ? DX - 1 : bx - 1, nw = bw == 0 ? DW - 1 : bw - 1;   // the places that were read last
        if (st + DX - 1 < stages) {
            load_rows(st + DX - 1, rows_at(nx));
            if (ONE)
                load_weights(st + DW - 1, weights_at(nx));
        }
        if (!ONE && st + DW - 1 < stages)
            load_weights(st + DW - 1, weights_at(nw));
        multiply(rows_at(bx), weights_at(ONE ? bx : bw), k - st * KC);
        bx = bx + 1 == DX ? 0 : bx + 1;
        bw = bw + 1 == DW ? 0 : bw + 1;
    }
    auto put = [&](int t, int group, f32x4 v) {
        put4<DT>(a, rows, rows.lo + (uint32_t)(t * 16 + q * 4), n0 + (uint32_t)(group * 16 + col), v);
    };
    if constexpr (KS == 1) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
            put(t, ns, acc[t]);
    } else {
        f32x4* joined = reinterpret_cast<f32x4*>(&rows_at(0));
        __syncthreads();
#pragma unroll
        for (int t = 0; t < TT; ++t)
            joined[((ns * TT + t) * KS + ks) * kWave + lane] = acc[t];
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
// wait for them. Half the start of k_gemm_fp4_stream (13 x 1000 x 2051: 7.2
// against 8.3 us), but 16 lines of the cache a load (16 x 8192 x 8192: 40 against 21).
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
    Coded<GR> w[D];
    Raw8<DT> xs[D][4];
    auto load = [&](int i, int d) {
        const int at = ks + i * KS, k0 = at * 128 + q * 8;
#pragma unroll
        for (int s = 0; s < 4; ++s)
            xs[d][s] = at * 128 + 128 <= k ? ld_raw8<DT, false>(xat, k0 + 32 * s, k) : ld_raw8<DT, true>(xat, k0 + 32 * s, k);
        w[d] = ld_coded<GR>(bat, sat, (uint32_t)at, kbytes, a.groups);
    };
    f32x4 acc[1] = {};
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (d < mine)
            load(d, d);
    for (int i = 0; i < mine; i += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (i + d >= mine)
                break;
            multiply_chunk<DT, GR, 1>(w[d], [&](int, int m) { return parts8<DT>(xs[d][m]); }, acc);
            if (i + d + D < mine)
                load(i + d + D, d);
        }
    }
    joined[ks][lane] = acc[0];
    __syncthreads();
    if (ks == 0) {
        f32x4 v = joined[0][lane];
#pragma unroll
        for (int s = 1; s < KS; ++s)
            v += joined[s][lane];
        put4<DT>(a, rows, rows.lo + (uint32_t)(q * 4), n0 + c, v);
    }
}

// Here, not later: the compiler would move sums to where they are next used, past the
// branches between, and hold all that they are made of until then.
template <int N>
__device__ __forceinline__ void keep(f32x4 (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+v"(x[i]));
}

// Many BF16 rows: 128 x 256 results a workgroup of 2 x 4 waves, one on a CU, 4 x 4
// products of 16 x 16 a wave, 128 of k a stage, one or two stages on their way. Steps of one
// row fragment: its products, and while the matrix cores run the fragment after
// the next is read, the next 32's weights are made (their values are exact in BF16),
// the scales join the sums of the step before, and a later stage asks for its share:
// all loads at once would hold the wave up for as long as the cache takes them. A stage
// is opened before the one before has ended, so that its first steps find their
// operands. 1024 x 8192 x 8192 with operands in the last-level cache: 118 to 122 us (1.13 to 1.17 PFLOP/s),
// 140 with stages one after the other, 160 in 128 x 128 tiles whose waves loaded their weights
// themselves; with operands from memory 128 to 133 (groups of 32: 171).
template <int GR>
__global__ __launch_bounds__(8 * kWave, 2) void k_gemm_fp4_tile(GemmFp4Args a)
{
    constexpr int TM = 4, TN = 4, WM = 2, WN = 4, NBUF = 3, KC = 128;
    constexpr int BM = 16 * TM * WM, BN = 16 * TN * WN, MG = GR / 32, SG = 4 / MG, kSteps = 4 * TM;
    using S = Stager<1, GR, BM, BN, BM, KC, WM * WN * kWave, true>;
    constexpr int kOpen = kSteps - S::N;   // the first step that may read the next stage
    static_assert(kOpen >= 0 && kOpen <= 2 * TM + TM - 1, "");
    __shared__ __align__(16) typename S::Stage ring[NBUF];
    static_assert(sizeof(ring) <= 160 * 1024, "");
    const int lane = lane_id(), wave = wave_id(), col = lane % 16, q = lane / 16;
    const Tiles tiles = count_tiles(a, BM);
    uint32_t tm, tn;
    if (!pick_tile(tiles, (a.n + BN - 1) / BN, tm, tn))
        return;
    const uint32_t n0 = tn * BN;
    const TileRows rows = find_tile(a, tiles, tm, BM);
    if (rows.lo >= rows.hi)
        return;
    if (rows.expert < 0) {
        zero_tile<1>(a, rows, n0, BN);
        return;
    }
    S s(a, rows, n0);
    const int stages = ((int)a.k + KC - 1) / KC;
    const int wm = wave / WN * TM * 16, wn = wave % WN * TN * 16;
    f32x4 acc[TM][TN] = {}, sum[TM][TN] = {};
    uint32_t code[2][TN];
    float by[2][TN] = {};
    bf16x8 b[2][TN], f[4];
    auto row = [&](int t) { return wn + t * 16 + col; };
    auto frag = [&](const typename S::Stage& st, int n) { return S::rows_of(st, wm + n % TM * 16 + col, n / TM * 32 + q * 8).p[0]; };
    auto scale = [&](int r) {
#pragma unroll
        for (int t = 0; t < TN; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[r][t][e] = __builtin_fmaf(sum[r][t][e], by[0][t], acc[r][t][e]);
        keep(acc[r]);
    };
    if (stages > 0) {
        unrolled<S::N>([&](auto i) { s.template load<i()>(0, ring[0]); });
        if (stages > 1)
            unrolled<S::N>([&](auto i) { s.template load<i()>(1, ring[1]); });
        open_stage<S::N>(stages > 1);
        f[0] = frag(ring[0], 0);
        f[1] = frag(ring[0], 1);
#pragma unroll
        for (int t = 0; t < TN; ++t) {
            code[0][t] = S::codes_of(ring[0], row(t), 0, q);
            code[1][t] = S::codes_of(ring[0], row(t), 1, q);
            by[1][t] = S::scale_of(ring[0], row(t), 0);
            b[0][t] = weights8(code[0][t]);
        }
    }
    int buf = 0;
    for (int st = 0; st < stages; ++st) {
        const typename S::Stage& now = ring[buf];
        buf = buf + 1 == NBUF ? 0 : buf + 1;
        const typename S::Stage& then = ring[buf];   // past the last one: anything, for nothing
        typename S::Stage& late = ring[buf + 1 == NBUF ? 0 : buf + 1];
        unrolled<kSteps>([&](auto step) {
            constexpr int n = step(), m = n / TM, r = n % TM, before = (n + kSteps - 1) % kSteps;   // before: its products are done
            if constexpr (n == kOpen)   // nothing but the next stage is on its way
                open_stage<0>(false);
            f[(n + 2) % 4] = n + 2 < kSteps ? frag(now, n + 2) : frag(then, n + 2 - kSteps);
#pragma unroll
            for (int t = 0; t < TN; ++t)
                sum[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[n % 4], b[m & 1][t],
                                                                    m % MG == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : sum[r][t], 0, 0, 0);
            if constexpr (n >= kOpen)
                if (st + 2 < stages)
                    s.template load<n - kOpen>(st + 2, late);
            if constexpr (before / TM % MG == MG - 1)
                scale(before % TM);
            // a share of the next weights
#pragma unroll
            for (int t = r * TN / TM; t < (r + 1) * TN / TM; ++t)
                b[(m + 1) & 1][t] = weights8(code[(m + 1) & 1][t]);
            if constexpr (r == TM - 1)
#pragma unroll
                for (int t = 0; t < TN; ++t)
                    code[m & 1][t] = m < 2 ? S::codes_of(now, row(t), m + 2, q) : S::codes_of(then, row(t), m - 2, q);
            if constexpr (r == 0 && m % MG == 0)   // the scales before have joined
#pragma unroll
                for (int t = 0; t < TN; ++t) {
                    by[0][t] = by[1][t];
                    if (m / MG + 1 < SG)
                        by[1][t] = S::scale_of(now, row(t), m / MG + 1);
                }
            if constexpr (n == kSteps - 3)
#pragma unroll
                for (int t = 0; t < TN; ++t)
                    by[1][t] = S::scale_of(then, row(t), 0);
            __builtin_amdgcn_sched_barrier(0);
        });
    }
    scale(TM - 1);
#pragma unroll
    for (int r = 0; r < TM; ++r)
#pragma unroll
        for (int t = 0; t < TN; ++t)
            put4<1>(a, rows, rows.lo + (uint32_t)(wm + r * 16 + q * 4), n0 + (uint32_t)(wn + t * 16 + col), acc[r][t]);
}

// Many FP32 rows: 64 x 128 results a workgroup of 2 x 2 waves, two on a CU, 2 x 4 products of
// 16 x 16 a wave (four channels to a fragment of three parts: with two, LDS would
// be as busy as the matrix cores), 128 of k a stage. The rows have one place in LDS and
// the next stage's wait in registers; the other workgroup computes while this one
// changes stages. 512 x 8192 x 8192: 190 us, three products at 1.08 PFLOP/s.
template <int GR>
__global__ __launch_bounds__(4 * kWave, 2) void k_gemm_fp4_parts(GemmFp4Args a)
{
    constexpr int DT = 0, TM = 2, TN = 4, WM = 2, WN = 2, KC = 128;
    constexpr int BM = 16 * TM * WM, BN = 16 * TN * WN, MG = GR / 32, P = 3, kSteps = 4 * TM;
    using S = Stager<DT, GR, BM, BN, BM, KC, WM * WN * kWave, false>;
    __shared__ __align__(16) typename S::Rows x;
    __shared__ __align__(16) typename S::Weights ring[2];
    static_assert(S::NXR + S::N <= kSteps && sizeof(x) + sizeof(ring) <= 80 * 1024, "");
    const int lane = lane_id(), wave = wave_id(), col = lane % 16, q = lane / 16;
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
    S s(a, rows, n0);
    const int stages = ((int)a.k + KC - 1) / KC;
    const int wm = wave / WN * TM * 16, wn = wave % WN * TN * 16;
    auto row = [&](int t) { return wn + t * 16 + col; };
    f32x4 acc[TM][TN] = {};
    if (stages > 0) {
        unrolled<S::NXR>([&](auto i) { s.template load_x<i()>(0); });
        order();
        unrolled<S::N>([&](auto i) { s.template load<i()>(0, ring[0]); });
    }
    for (int st = 0; st < stages; ++st) {
        const typename S::Weights& now = ring[st & 1];
        typename S::Weights& late = ring[st & 1 ^ 1];
        order();
        __builtin_amdgcn_s_barrier();   // the stage before has been read
        order();
        s.store_x(x);
        open_stage<0>(false);
        uint32_t code[2][TN];
        float by[2][TN];
        bf16x8 b[2][TN];
        f32x4 sum[TM][TN];
        Parts8<DT> f[3];
        auto frag = [&](int n) { return S::rows_of(x, wm + n % TM * 16 + col, n / TM * 32 + q * 8); };
        auto scale = [&](int r, int g) {
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[r][t][e] = __builtin_fmaf(sum[r][t][e], by[g & 1][t], acc[r][t][e]);
            keep(acc[r]);
        };
        f[0] = frag(0);
        f[1] = frag(1);
#pragma unroll
        for (int t = 0; t < TN; ++t) {
            code[0][t] = S::codes_of(now, row(t), 0, q);
            code[1][t] = S::codes_of(now, row(t), 1, q);
            by[0][t] = S::scale_of(now, row(t), 0);
            b[0][t] = weights8(code[0][t]);
        }
        unrolled<kSteps>([&](auto step) {
            constexpr int n = step(), m = n / TM, r = n % TM, before = n - 1;   // before: its products are done
            if constexpr (n + 2 < kSteps)
                f[(n + 2) % 3] = frag(n + 2);
#pragma unroll
            for (int p = P - 1; p >= 0; --p)
#pragma unroll
                for (int t = 0; t < TN; ++t) {
                    const bool first = m % MG == 0 && p == P - 1;
                    sum[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[n % 3].p[p], b[m & 1][t],
                                                                        first ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : sum[r][t], 0, 0, 0);
                }
            if (st + 1 < stages) {
                if constexpr (n < S::NXR)
                    s.template load_x<n>(st + 1);
                else if constexpr (n - S::NXR < S::N)
                    s.template load<n - S::NXR>(st + 1, late);
            }
            if constexpr (before >= 0 && before / TM % MG == MG - 1)
                scale(before % TM, before / TM / MG);
            if constexpr (m < 3)   // a share of the next weights
#pragma unroll
                for (int t = r * TN / TM; t < (r + 1) * TN / TM; ++t)
                    b[(m + 1) & 1][t] = weights8(code[(m + 1) & 1][t]);
            if constexpr (r == TM - 1 && m < 2)
#pragma unroll
                for (int t = 0; t < TN; ++t)
                    code[m & 1][t] = S::codes_of(now, row(t), m + 2, q);
            if constexpr (r == 0 && m % MG == 0 && m + MG < 4)   // the scales before this group's have joined
#pragma unroll
                for (int t = 0; t < TN; ++t)
                    by[(m / MG + 1) & 1][t] = S::scale_of(now, row(t), m / MG + 1);
            __builtin_amdgcn_sched_barrier(0);
        });
        scale(TM - 1, 3 / MG);
    }
#pragma unroll
    for (int r = 0; r < TM; ++r)
#pragma unroll
        for (int t = 0; t < TN; ++t)
            put4<DT>(a, rows, rows.lo + (uint32_t)(wm + r * 16 + q * 4), n0 + (uint32_t)row(t), acc[r][t]);
}

// A call's workgroups: whole rounds of the XCDs for the tiles with an expert and
// for those without.
inline hipError_t launch_grid(GemmFp4Args& a, const void* fn, const char* name, size_t bm, size_t bn, unsigned threads, hipStream_t s)
{
    void* params[] = {&a};
    const size_t grid = (row_tiles(a, bm) * ((a.n + bn - 1) / bn) + 2 * kXcds) / kXcds * kXcds;
    return launch_logged(name, fn, dim3((unsigned)grid), dim3(threads), params, s);
}

template <int DT, int GR, int TT, int TR, int KS, int NS, int KC, int DX, int DW, bool WHOLE>
hipError_t launch_stream(GemmFp4Args& a, const char* name, hipStream_t s)
{
    return launch_grid(a, (const void*)k_gemm_fp4_stream<DT, GR, TT, TR, KS, NS, KC, DX, DW, WHOLE>, name, 16 * TT,
                       16 * NS, KS * NS * kWave, s);
}

// A kind of workgroup: its tile, how many a CU takes, and the microseconds that
// 1024 of k take it alone on its CU, and with the CU full.
struct Kind {
    double bm, bn, per_cu, alone, full;
};

// Estimated time. The kinds' figures are measured at 8192 and 4096 of k, with
// groups of 128 (32: 5 to 35% more, alike for all) and weights in the last-level cache. CUs that
// are full, round by round, and a last round that fills up from `alone` to `full`.
// Up to four rows two workgroups of 16 x 32 do share a CU, which `per_cu` leaves out: beyond
// two rounds of them it estimates too much.
inline double estimate(const GemmFp4Args& a, const Kind& x, double rows)
{
    const double cus = device_cu_count();
    double tm = (double)(long long)((rows + x.bm - 1.0) / x.bm);
    if (a.offsets) {   // about half a tile of each expert is empty
        const double owners = (double)a.experts < rows ? (double)a.experts : rows;
        tm = rows / x.bm + 0.5 * owners;
        tm = tm < owners ? owners : tm;
    }
    const double tn = (double)((a.n + (size_t)x.bn - 1) / (size_t)x.bn), t = tm * tn / cus, k = a.k / 1024.0, start = 0.5;
    if (((double)row_tiles(a, (size_t)x.bm) * tn + 16.0) * 512.0 >= 4294967296.0)
        return 1e300;   // threads of one launch
    const double rounds = (double)(long long)(t / x.per_cu), rest = t - rounds * x.per_cu;
    double time = rounds * (start + k * x.full);
    if (rest > 0.0)
        time += start + k * (rest > 1.0 ? x.alone + (x.full - x.alone) * (rest - 1.0) / (x.per_cu - 1.0) : x.alone);
    return time;
}

// Rows that no expert has are only known on the device: as if all, and as if half had one.
inline double estimate(const GemmFp4Args& a, const Kind& x)
{
    const double all = estimate(a, x, (double)a.rows);
    return a.offsets ? 0.5 * (all + estimate(a, x, 0.5 * (double)a.rows)) : all;
}

// The kinds, and where another would go wrong (us, groups of 128; dense ones with weights in the
// last-level cache and, behind the stroke, from memory, where those of 64 experts are always):
//   BF16                          16x16     16x32     16x64     32x32     32x128    64x32     64x128    128x256
//   1 x 1024 x 8192               6.6/6.7   8.8/8.8
//   1 x 6144 x 8192               8.8/9.7   8.8/9.9   23/30
//   1 x 8192 x 8192               9.1/10.4  9.4/10.4  24/29
//   1 x 14336 x 4096              9.4/11.0  7.4/9.4   13/17
//   1 x 14336 x 8192              16/18     14/16     24/31
//   1 x 28672 x 4096              16/18     15/16     15/18               18/24               27/28
//   1 x 28672 x 8192              26/30     24/28     28/35               33/47               51/53
//   13 x 4096 x 8192              8.6/9.5   10.2/11.4
//   16 x 8192 x 8192              15/17     11.2/12.6 23/29
//   32 x 1024 x 8192              8.2/8.3   10/10               14/14
//   32 x 6144 x 8192              22/24     19/21     24/30     14/15     32/46
//   32 x 8192 x 8192              28/31     19/21     24/29     14/16     32/43
//   32 x 14336 x 8192             48/52     36/39     27/32     27/28     32/46     39/41
//   32 x 28672 x 8192             94/101    63/68     42/58     52/54     34/49     77/79     51/57
//   64 x 8192 x 8192                                                                22/24     50/56
//   64 x 4096 x 4096                                            8.6/9.4             11.6/12.4
//   128 x 8192 x 8192                                                     32/41     41/42     50/55     102/111
//   512 x 8192 x 8192                                                               158/162   88/96     104/111
//   1024 x 8192 x 8192                                                                        171/179   120/128
// (28672 channels of one row get 32 x 128, the one choice here that is wrong by more than a tenth.)
//   64 experts x 4 x 4096 x 4096            190       120
//   64 experts x 24 x 4096 x 4096                               270       162                 231       269
//   64 experts x 48 x 4096 x 4096                                         254       415       252       276
//   64 experts x 256 x 4096 x 4096                                                            805       580
//   FP32                            few       16x32     16x64     32x128    64x128 parts
//   13 x 1000 x 2051                7.2/7.4   8.3/8.2
//   16 x 8192 x 8192                40/41     21/23
//   128 x 8192 x 8192                                             71/73     137/139
//   512 x 8192 x 8192                                             234/236   188/194
//   64 experts x 4 x 4096 x 4096            296       180
//   12 experts x 129 x 2100 x 2056                              67        85
//   64 experts x 48 x 4096 x 4096                               481       397
template <int DT, int GR>
hipError_t launch_fp4(const GemmFp4Args& in, hipStream_t s)
{
    GemmFp4Args a = in;
    constexpr Kind kBf16[] = {{16, 32, 1, 1.05, 1.05}, {16, 64, 4, 2.6, 7.5}, {32, 32, 1, 1.6, 1.6}, {32, 128, 2, 3.5, 9.5},
                              {64, 32, 1, 2.3, 2.3}, {64, 128, 2, 6.2, 11.8}, {128, 256, 1, 13.8, 15.0},
                              {16, 16, 1, 0.6, 0.6}};
    constexpr Kind kFp32[] = {{16, 32, 1, 2.2, 2.2}, {16, 64, 2, 4.3, 5.6}, {32, 128, 2, 9.0, 15.1}, {64, 128, 2, 16.7, 23.8},
                              {16, 16, 1, 2.0, 2.0}};
    const bool whole = DT == 1 && (uintptr_t)a.a % 16 == 0 && a.ld_a % 8 == 0 && a.k % 8 == 0;
    const Kind* kinds = DT == 0 ? kFp32 : kBf16;
    const int n = DT == 0 ? 5 : whole ? 8 : 6;   // rows by way of registers have no larger tile: 1024 x 8192 x 8191 takes 190 us
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
        case 0: return launch_stream<0, GR, 1, 16, 4, 2, 512, 2, 2, false>(a, "k_gemm_fp4_stream 16x32", s);
        case 1: return launch_stream<0, GR, 1, 16, 1, 4, 256, 2, 2, false>(a, "k_gemm_fp4_stream 16x64", s);
        case 2: return launch_stream<0, GR, 2, 32, 1, 8, 128, 2, 2, false>(a, "k_gemm_fp4_stream 32x128", s);
        case 3: return launch_grid(a, (const void*)k_gemm_fp4_parts<GR>, "k_gemm_fp4_parts", 64, 128, 4 * kWave, s);
        default: return launch_grid(a, (const void*)k_gemm_fp4_few<0, GR>, "k_gemm_fp4_few", 16, 16, 8 * kWave, s);
        }
    } else if (whole) {
        const bool four = a.rows <= 4;   // fewer rows to load: 4 x 8192 x 8192 9.4 us, 10.3 from memory; 5 rows 10.6 and 11.4
        switch (best) {
        case 0: return four ? launch_stream<1, GR, 1, 4, 4, 2, 1024, 3, 3, true>(a, "k_gemm_fp4_stream 16x32, four rows", s) : launch_stream<1, GR, 1, 16, 4, 2, 1024, 3, 3, true>(a, "k_gemm_fp4_stream 16x32", s);
        case 1: return launch_stream<1, GR, 1, 16, 1, 4, 256, 2, 2, true>(a, "k_gemm_fp4_stream 16x64", s);
        case 2: return launch_stream<1, GR, 2, 32, 4, 2, 512, 3, 3, true>(a, "k_gemm_fp4_stream 32x32", s);
        case 3: return launch_stream<1, GR, 2, 32, 1, 8, 256, 2, 2, true>(a, "k_gemm_fp4_stream 32x128", s);
        case 4: return launch_stream<1, GR, 4, 64, 4, 2, 512, 2, 3, true>(a, "k_gemm_fp4_stream 64x32", s);
        case 5: return launch_stream<1, GR, 4, 64, 1, 8, 128, 3, 3, true>(a, "k_gemm_fp4_stream 64x128", s);
        case 6: return launch_grid(a, (const void*)k_gemm_fp4_tile<GR>, "k_gemm_fp4_tile", 128, 256, 8 * kWave, s);
        default: return four ? launch_stream<1, GR, 1, 4, 8, 1, 1024, 4, 4, true>(a, "k_gemm_fp4_stream 16x16, four rows", s) : launch_stream<1, GR, 1, 16, 8, 1, 1024, 3, 4, true>(a, "k_gemm_fp4_stream 16x16", s);
        }
    } else {
        switch (best) {
        case 0: return launch_stream<1, GR, 1, 16, 4, 2, 1024, 3, 3, false>(a, "k_gemm_fp4_stream 16x32, rows by way of registers", s);
        case 1: return launch_stream<1, GR, 1, 16, 1, 4, 256, 2, 2, false>(a, "k_gemm_fp4_stream 16x64, rows by way of registers", s);
        case 2: return launch_stream<1, GR, 2, 32, 4, 2, 512, 3, 3, false>(a, "k_gemm_fp4_stream 32x32, rows by way of registers", s);
        case 3: return launch_stream<1, GR, 2, 32, 1, 8, 256, 2, 2, false>(a, "k_gemm_fp4_stream 32x128, rows by way of registers", s);
        case 4: return launch_stream<1, GR, 4, 64, 4, 2, 512, 2, 2, false>(a, "k_gemm_fp4_stream 64x32, rows by way of registers", s);
        default: return launch_stream<1, GR, 4, 64, 1, 8, 128, 3, 3, false>(a, "k_gemm_fp4_stream 64x128, rows by way of registers", s);
        }
    }
}

}  // namespace
}  // namespace rx
