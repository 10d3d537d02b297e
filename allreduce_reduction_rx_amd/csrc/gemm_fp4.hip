// gemm_fp4.hip -- rows to 4-bit floating point with a scale for each group, and
// the product of activations with such weights, dense or grouped by expert
// (gfx950). Defined in rx.h.
#include "expert_tiles.hpp"

namespace rx {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// A group's scale and multiplier from its absmax A, as i8_scale() with 6 for 127.
__device__ __forceinline__ void fp4_scale(float a, float& s, float& r)
{
    const float sv = a / 6.0f, rv = 6.0f / a;
    const bool degenerate = (a == 0.0f) | (sv == 0.0f) | !__builtin_isfinite(rv);
    const bool finite = __builtin_isfinite(a);
    s = !finite ? a : degenerate ? 1.0f : sv;
    r = !finite ? 0.0f : degenerate ? 1.0f : rv;
}

// A workgroup a row, a lane a vector: 4 to 32 neighbouring lanes have a group.
template <int DT, bool TAIL>
__global__ __launch_bounds__(256) void k_quant_fp4(QuantFp4Args a)
{
    constexpr int VE = Elem<DT>::kVE;
    const size_t t = blockIdx.x;
    const int k = (int)a.k, nvec = (k + VE - 1) / VE, lanes = a.group / VE;
    const size_t groups = (a.k + a.group - 1) / a.group;
    const void* row = static_cast<const char*>(a.x) + t * a.ld_x * Elem<DT>::kBytes;
    for (int v0 = 0; v0 < nvec; v0 += (int)blockDim.x) {
        const int v = v0 + (int)threadIdx.x;
        const u32x4 x = ld_row<DT, TAIL, true>(row, v < nvec ? v : nvec - 1, k);
        float s, r;
        fp4_scale(bits_f32(group_max_rt(v < nvec ? vec_absmax<DT>(x) : 0, lanes)), s, r);
        if (v >= nvec)
            continue;
        if (v % lanes == 0)
            a.scales[t * groups + v / lanes] = s;
        float f[VE];
        unpack<DT>(x, f);
        uint32_t q = 0;
#pragma unroll
        for (int i = 0; i < VE; ++i)
            f[i] = r == 0.0f ? 0.0f : f[i] * r;   // a NaN's product has no code
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[0], f[1], 1.0f, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[2], f[3], 1.0f, 1);
        if constexpr (VE == 8) {
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[4], f[5], 1.0f, 2);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[6], f[7], 1.0f, 3);
        }
        uint8_t* p = a.codes + t * a.ld_codes + (size_t)v * (VE / 2);
        const int left = k - v * VE;
        if (!TAIL || left >= VE) {
            if constexpr (VE == 8)
                *reinterpret_cast<u32_any*>(p) = q;
            else
                *reinterpret_cast<u16_any*>(p) = (uint16_t)q;
        } else {
            for (int b = 0; b < (left + 1) / 2; ++b)
                p[b] = (uint8_t)(q >> (8 * b));
        }
    }
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------

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

// Few rows: 16 TT rows x 16 NT NS channels a workgroup of KS x NS waves. A wave
// has 16 NT channels and every KS-th chunk of 128 of k; the KS sums meet in LDS
// in their order. Weights go from memory to registers, D chunks ahead, and to
// BF16 there (their values are exact); rows come from the caches.
template <int DT, int GR, int TT, int NT, int KS, int NS>
__global__ __launch_bounds__(KS * NS * kWave) void k_gemm_fp4_few(GemmFp4Args a)
{
    constexpr int BM = 16 * TT, BN = 16 * NT * NS, SG = 128 / GR, EB = Elem<DT>::kBytes;
    constexpr int D = 4, XD = (DT == 1 ? TT <= 2 : TT <= 1) ? 2 : 1;
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
    u32x4 cw[D][NT];
    float sc[D][NT][SG];
    Raw8<DT> xs[XD][TT][4];
    auto chunk = [&](int i) { return ks + i * KS; };
    auto load = [&](int i, int d) {
        const uint32_t c = (uint32_t)chunk(i);
        uint32_t byte = c * 64 + (uint32_t)q * 16;
        byte = byte < kbytes ? byte : 0;   // met by zeros of a
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            cw[d][t] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(bbase + (bfrom[t] + byte)));
#pragma unroll
            for (int g = 0; g < SG; ++g) {
                const uint32_t at = c * SG + g;
                sc[d][t][g] = sbase[sfrom[t] + (at < a.groups ? at : a.groups - 1)];
            }
        }
    };
    auto load_x = [&](int i, int d) {
        const int k0 = chunk(i) * 128 + q * 8;
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (chunk(i) * 128 + 128 <= k)
                    xs[d][t][s] = ld_raw8<DT, false>(xbase + xfrom[t], k0 + 32 * s, k);
                else
                    xs[d][t][s] = ld_raw8<DT, true>(xbase + xfrom[t], k0 + 32 * s, k);
            }
    };
    f32x4 acc[TT][NT] = {};
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (d < mine)
            load(d, d);
    if (XD > 1 && mine > 0)
        load_x(0, 0);
    for (int i = 0; i < mine; i += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (i + d >= mine)
                break;
            if (XD == 1)
                load_x(i + d, 0);
            else if (i + d + 1 < mine)
                load_x(i + d + 1, (d + 1) % XD);
            u32x4 w[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
                w[t] = turned(cw[d][t]);
            float s[NT][SG];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int g = 0; g < SG; ++g)
                    s[t][g] = sc[d][t][g];
            if (i + d + D < mine)
                load(i + d + D, d);
#pragma unroll
            for (int g = 0; g < SG; ++g) {
                f32x4 sum[TT][NT] = {};
#pragma unroll
                for (int m = g * (4 / SG); m < (g + 1) * (4 / SG); ++m) {
                    bf16x8 b[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        b[t] = weights8(w[t][m]);
#pragma unroll
                    for (int r = 0; r < TT; ++r) {
                        const Parts8<DT> x = parts8<DT>(xs[d % XD][r][m]);
#pragma unroll
                        for (int p = DT == 0 ? 2 : 0; p >= 0; --p)
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                sum[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.p[p], b[t], sum[r][t], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int r = 0; r < TT; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[r][t][e] = __builtin_fmaf(sum[r][t][e], s[t][g], acc[r][t][e]);
            }
        }
    }
    // a lane has rows 4 q .. 4 q + 3 of channel `col`
    auto put = [&](int r, int t, int group, f32x4 v) {
        const uint32_t n = n0 + (uint32_t)((group * NT + t) * 16 + col);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t m = rows.lo + (uint32_t)(r * 16 + q * 4 + e);
            if (m < rows.hi && n < a.n) {
                char* p = static_cast<char*>(a.out) + ((size_t)m * a.ld_out + n) * EB;
                if constexpr (DT == 0)
                    *reinterpret_cast<float*>(p) = v[e];
                else
                    *reinterpret_cast<uint16_t*>(p) = (uint16_t)pack_bf16(v[e], 0.0f);
            }
        }
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
            for (int w = 1; w < KS; ++w)
                v += joined[i * KS + w][lane];
            put(i / NT % TT, i % NT, i / (NT * TT), v);
        }
    }
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

template <int DT, int GR, int TT>
hipError_t launch_rows(GemmFp4Args& a, hipStream_t s)
{
    const size_t tiles = row_tiles(a, 16 * TT), cus = (size_t)device_cu_count();
    auto fills = [&](size_t bn) { return tiles * ((a.n + bn - 1) / bn) >= cus; };
    return fills(256) ? launch_few<DT, GR, TT, 2, 1>(a, s)
           : fills(64) ? launch_few<DT, GR, TT, 2, 4>(a, s)
           : fills(32) ? launch_few<DT, GR, TT, 2, 8>(a, s)
                       : launch_few<DT, GR, TT, 1, 8>(a, s);
}

template <int DT, int GR>
hipError_t launch_group(GemmFp4Args& a, hipStream_t s)
{
    const size_t owners = a.offsets ? ((size_t)a.experts < a.rows ? (size_t)a.experts : a.rows) : 1;
    const size_t mean = (a.rows + owners - 1) / owners;
    return mean <= 16 ? launch_rows<DT, GR, 1>(a, s) : mean <= 32 ? launch_rows<DT, GR, 2>(a, s) : launch_rows<DT, GR, 4>(a, s);
}

}  // namespace

hipError_t launch_quant_fp4(const QuantFp4Args& in, int dtype, hipStream_t s)
{
    QuantFp4Args a = in;
    void* params[] = {&a};
    const bool tail = partial(a.k, dtype);
    const void* fn = dtype == 0 ? tail ? (const void*)k_quant_fp4<0, true> : (const void*)k_quant_fp4<0, false>
                     : tail     ? (const void*)k_quant_fp4<1, true>
                                : (const void*)k_quant_fp4<1, false>;
    return launch_logged("k_quant_fp4", fn, dim3((unsigned)a.rows), dim3(threads_for(vectors(a.k, dtype), 256)), params, s);
}

hipError_t launch_gemm_fp4(const GemmFp4Args& in, int dtype, hipStream_t s)
{
    GemmFp4Args a = in;
    if (dtype == 0)
        return a.group == 32 ? launch_group<0, 32>(a, s) : a.group == 64 ? launch_group<0, 64>(a, s) : launch_group<0, 128>(a, s);
    return a.group == 32 ? launch_group<1, 32>(a, s) : a.group == 64 ? launch_group<1, 64>(a, s) : launch_group<1, 128>(a, s);
}

}  // namespace rx
