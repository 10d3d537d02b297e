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

// Few rows: 16 TT rows x 16 NT NS channels a workgroup of KS x NS waves. A wave
// has 16 NT channels and every KS-th chunk of 128 of k; the KS sums meet in LDS
// in their order. Weights go from memory to registers, D chunks ahead, and to
// BF16 there (their values are exact). The rows come from the caches, as far
// ahead and before the weights: loads return in order, so a row's chunk that
// was asked for after the weights would wait for them.
template <int DT, int GR, int TT, int NT, int KS, int NS>
__global__ __launch_bounds__(KS * NS * kWave) void k_gemm_fp4_few(GemmFp4Args a)
{
    constexpr int BM = 16 * TT, BN = 16 * NT * NS, EB = Elem<DT>::kBytes;
    constexpr int D = DT == 1 ? TT == 1 ? 4 : TT == 2 ? 3 : 2 : TT == 1 ? 3 : 2;
    __shared__ f32x4 joined[KS > 1 ? NS * KS * TT * NT : 1][KS > 1 ? kWave : 1];
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
    const int k = (int)a.k, chunks = (k + 127) / 128, mine = chunks > ks ? (chunks - ks + KS - 1) / KS : 0;
    const uint32_t kbytes = (uint32_t)(k + 31) / 32 * 16;
    const char* xbase = static_cast<const char*>(a.a) + (size_t)rows.lo * a.ld_a * EB;
    const uint8_t* bbase = a.b + (size_t)rows.expert * a.stride_b + (size_t)n0 * a.ld_b;
    const float* sbase = a.b_scales + ((size_t)rows.expert * a.n + n0) * a.groups;
    uint32_t xfrom[TT], bfrom[NT], sfrom[NT];   // below 2^32: 64 rows of a stride below 2^23 elements
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        const uint32_t r = (uint32_t)(i * 16 + col), most = rows.hi - 1 - rows.lo;
        xfrom[i] = (r < most ? r : most) * (uint32_t)a.ld_a * EB;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const uint32_t r = (uint32_t)((ns * NT + i) * 16 + col), most = a.n - 1 - n0, at = r < most ? r : most;
        bfrom[i] = at * (uint32_t)a.ld_b;
        sfrom[i] = at * a.groups;
    }
    Coded<GR> w[D][NT];
    Raw8<DT> xs[D][TT][4];
    auto load = [&](int i, int d) {
        const int c = ks + i * KS, k0 = c * 128 + q * 8;
        if (c * 128 + 128 <= k) {
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    xs[d][t][s] = ld_raw8<DT, false>(xbase + xfrom[t], k0 + 32 * s, k);
        } else {
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    xs[d][t][s] = ld_raw8<DT, true>(xbase + xfrom[t], k0 + 32 * s, k);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
            w[d][t] = ld_coded<GR>(bbase + bfrom[t], sbase + sfrom[t], (uint32_t)c, kbytes, a.groups);
    };
    f32x4 acc[TT][NT] = {};
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (d < mine)
            load(d, d);
    for (int i = 0; i < mine; i += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (i + d >= mine)
                break;
            multiply_chunk<DT, GR, TT, NT>(w[d], [&](int r, int m) { return parts8<DT>(xs[d][r][m]); }, acc);
            if (i + d + D < mine)
                load(i + d + D, d);
        }
    }
    auto put = [&](int r, int t, int group, f32x4 v) {
        put4<DT>(a, rows, rows.lo + (uint32_t)(r * 16 + q * 4), n0 + (uint32_t)((group * NT + t) * 16 + col), v);
    };
    if constexpr (KS == 1) {
#pragma unroll
        for (int r = 0; r < TT; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                put(r, t, ns, acc[r][t]);
    } else {
#pragma unroll
        for (int r = 0; r < TT; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                joined[((ns * TT + r) * NT + t) * KS + ks][lane] = acc[r][t];
        __syncthreads();
        for (int i = wave; i < NS * TT * NT; i += KS * NS) {
            f32x4 v = joined[i * KS][lane];
#pragma unroll
            for (int s = 1; s < KS; ++s)
                v += joined[i * KS + s][lane];
            put(i / NT % TT, i % NT, i / (NT * TT), v);
        }
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

template <int DT, int GR, int TT, int NT, int KS>
hipError_t launch_few(GemmFp4Args& a, hipStream_t s)
{
    constexpr int NS = 8 / KS, BN = 16 * NT * NS;
    void* params[] = {&a};
    const size_t grid = (row_tiles(a, 16 * TT) * ((a.n + BN - 1) / BN) + 2 * kXcds) / kXcds * kXcds;
    return launch_logged("k_gemm_fp4_few", (const void*)k_gemm_fp4_few<DT, GR, TT, NT, KS, NS>, dim3((unsigned)grid),
                         dim3(8 * kWave), params, s);
}

template <int DT, int GR, int TM, int TN, int WM, int WN>
hipError_t launch_tile(GemmFp4Args& a, hipStream_t s)
{
    constexpr int BM = 16 * TM * WM, BN = 16 * TN * WN;
    void* params[] = {&a};
    const size_t grid = (row_tiles(a, BM) * ((a.n + BN - 1) / BN) + 2 * kXcds) / kXcds * kXcds;
    const void* fn = (const void*)k_gemm_fp4_tile<DT, GR, TM, TN, WM, WN, false>;
    if constexpr (DT == 1)
        if ((uintptr_t)a.a % 16 == 0 && a.ld_a % 8 == 0)
            fn = (const void*)k_gemm_fp4_tile<DT, GR, TM, TN, WM, WN, true>;
    return launch_logged("k_gemm_fp4_tile", fn, dim3((unsigned)grid), dim3(WM * WN * kWave), params, s);
}

template <int DT, int GR, int TT>
hipError_t launch_rows(GemmFp4Args& a, hipStream_t s)
{
    constexpr int NT = (DT == 0 ? 2 : 1) * TT >= 4 ? 1 : 2;   // what fits the registers
    const size_t tiles = row_tiles(a, 16 * TT), cus = (size_t)device_cu_count();
    auto fills = [&](size_t bn) { return tiles * ((a.n + bn - 1) / bn) >= cus; };
    return fills(128 * NT)          ? launch_few<DT, GR, TT, NT, 1>(a, s)
           : NT == 1 || fills(32)   ? launch_few<DT, GR, TT, NT, 8>(a, s)
                                    : launch_few<DT, GR, TT, 1, 8>(a, s);
}

template <int DT, int GR>
hipError_t launch_fp4(const GemmFp4Args& in, hipStream_t s)
{
    GemmFp4Args a = in;
    const size_t owners = a.offsets ? ((size_t)a.experts < a.rows ? (size_t)a.experts : a.rows) : 1;
    const size_t mean = (a.rows + owners - 1) / owners;
    if (mean > 64) {
        if constexpr (DT == 1)
            return launch_tile<DT, GR, 4, 4, 2, 2>(a, s);
        else
            return launch_tile<DT, GR, 4, 2, 1, 4>(a, s);
    }
    if (mean <= 16)
        return launch_rows<DT, GR, 1>(a, s);
    if constexpr (DT == 1)
        if (mean > 32)
            return launch_rows<DT, GR, 4>(a, s);
    return launch_rows<DT, GR, 2>(a, s);
}

}  // namespace
}  // namespace rx
