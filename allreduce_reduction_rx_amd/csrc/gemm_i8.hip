// gemm_i8.hip -- rows to 8-bit integers with a scale each, and the product of
// such matrices with a scale per token and channel, dense or grouped by
// expert (gfx950). Defined in rx.h.
#include "block_common.hpp"

namespace rx {
namespace {

template <int DT, bool TAIL>
__global__ __launch_bounds__(256) void k_quant_i8(QuantI8Args a)
{
    __shared__ uint32_t lds[4];
    const int tid = threadIdx.x, bd = blockDim.x;
    const size_t t = blockIdx.x;
    const int k = (int)a.k;
    const int nvec = (k + Elem<DT>::kVE - 1) / Elem<DT>::kVE;
    const void* row = static_cast<const char*>(a.x) + t * a.ld_x * Elem<DT>::kBytes;
    uint32_t m = 0;
    for (int v = tid; v < nvec; v += bd)
        m = umax(m, vec_absmax<DT>(ld_row<DT, TAIL>(row, v, k)));
    m = group_max<kWave>(m);
    if (bd > kWave) {
        if (lane_id() == 0)
            lds[tid / kWave] = m;
        __syncthreads();
        for (int w = 0; w < bd / kWave; ++w)
            m = umax(m, lds[w]);
    }
    float s, r;
    i8_scale(bits_f32(m), s, r);
    if (tid == 0)
        a.scales[t] = s;
    char* out = static_cast<char*>(a.codes) + t * a.ld_codes;
    for (int v = tid; v < nvec; v += bd) {
        uint32_t q[2];
        i8_codes<DT>(ld_row<DT, TAIL>(row, v, k), r, q);
        st_codes<DT, TAIL>(out, v, k, q);
    }
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

constexpr int kStep = 128;   // bytes of k in one stage: a row is one 128-byte line

// The rows [lo, hi) of tile `tm` (BM rows) and their expert. Each expert's
// rows start a tile of their own; past the last, tiles of the rows that no
// expert owns have expert -1. Every wave computes it for itself.
struct TileRows {
    uint32_t lo, hi;
    int expert;
};

__device__ __forceinline__ TileRows find_tile(const GemmI8Args& a, uint32_t tm, uint32_t bm)
{
    if (!a.offsets) {
        const uint32_t lo = tm * bm;
        return {lo, lo + bm < a.rows ? lo + bm : a.rows, 0};
    }
    const int lane = lane_id();
    uint32_t base = 0, end = 0;
    for (int e0 = 0; e0 < a.experts; e0 += kWave) {
        const int e = e0 + lane;
        uint32_t lo = 0, hi = 0;
        if (e < a.experts) {
            const int o0 = a.offsets[e], o1 = a.offsets[e + 1];
            lo = o0 < 0 ? 0 : (uint32_t)o0 < a.rows ? (uint32_t)o0 : a.rows;
            hi = o1 < 0 ? 0 : (uint32_t)o1 < a.rows ? (uint32_t)o1 : a.rows;
            hi = hi > lo ? hi : lo;
        }
        const uint32_t tiles = (hi - lo + bm - 1) / bm;
        uint32_t incl = tiles;
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const uint32_t o = __shfl_up(incl, d);
            if (lane >= d)
                incl += o;
        }
        const uint64_t past = __ballot(base + incl > tm);
        if (past) {
            const int l = __builtin_ctzll(past);
            const uint32_t first = base + (uint32_t)__builtin_amdgcn_readlane((int)(incl - tiles), l);
            const uint32_t rlo = (uint32_t)__builtin_amdgcn_readlane((int)lo, l) + (tm - first) * bm;
            const uint32_t rhi = (uint32_t)__builtin_amdgcn_readlane((int)hi, l);
            return {rlo, rlo + bm < rhi ? rlo + bm : rhi, e0 + l};
        }
        base += (uint32_t)__builtin_amdgcn_readlane((int)incl, kWave - 1);
        end = (uint32_t)__builtin_amdgcn_readlane((int)hi, (a.experts - e0 < kWave ? a.experts - e0 : kWave) - 1);
    }
    const uint32_t lo = end + (tm - base) * bm;
    return {lo < a.rows ? lo : a.rows, lo + bm < a.rows ? lo + bm : a.rows, -1};
}

template <int DT>
__device__ __forceinline__ void st_out(const GemmI8Args& a, size_t m, uint32_t n, float v)
{
    if constexpr (DT == 0)
        static_cast<float*>(a.out)[m * a.ld_out + n] = v;
    else
        static_cast<uint16_t*>(a.out)[m * a.ld_out + n] = (uint16_t)pack_bf16(v, 0.0f);
}

template <int DT>
__device__ void zero_tile(const GemmI8Args& a, const TileRows& r, uint32_t n0, uint32_t bn)
{
    for (uint32_t m = r.lo; m < r.hi; ++m)
        for (uint32_t n = n0 + threadIdx.x; n < n0 + bn && n < a.n; n += blockDim.x)
            st_out<DT>(a, m, n, 0.0f);
}

// 16 bytes of which only the first `nb` count (nb may be negative or large).
__device__ __forceinline__ i32x4 mask_bytes(i32x4 x, int nb)
{
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int r = nb - 4 * d;
        x[d] = r >= 4 ? x[d] : r <= 0 ? 0 : x[d] & ((1 << (8 * r)) - 1);
    }
    return x;
}

// 128 x 128 outputs, 4 waves of 64 x 64. Stages of 128 bytes of k go from
// global memory to LDS directly (16 bytes a lane, LDS written in lane
// order), the next one while this one is multiplied. Chunk c of row r sits
// at position c ^ (r & 7) of the row, so the 8 rows that one pass of a
// 16-byte read touches lie in different banks; the load picks its global
// chunk to match. Rows past the end read the last row, chunks past k read
// chunk 0 and are masked out of `a` in the last stage.
template <int DT>
__global__ __launch_bounds__(256) void k_gemm_i8(GemmI8Args a)
{
    constexpr int BM = 128, BN = 128;
    __shared__ __align__(16) int8_t lds[2][(BM + BN) * kStep];
    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const uint32_t ntn = (a.n + BN - 1) / BN;
    const uint32_t tm = blockIdx.x / ntn, n0 = (blockIdx.x % ntn) * BN;
    const TileRows rows = find_tile(a, tm, BM);
    if (rows.lo >= rows.hi)
        return;
    if (rows.expert < 0) {
        zero_tile<DT>(a, rows, n0, BN);
        return;
    }
    const int8_t* b = a.b + (size_t)rows.expert * a.stride_b;
    const int stages = (int)((a.k + kStep - 1) / kStep);

    auto load = [&](int st, int buf) {
#pragma unroll
        for (int i = 0; i < (BM + BN) * 8 / 256; ++i) {
            const int slot = i * 256 + wave * kWave + lane;     // 16-byte slots: row slot / 8
            const int r = slot / 8, c = (slot % 8) ^ (r & 7);
            uint32_t kk = (uint32_t)st * kStep + (uint32_t)c * 16;
            if (kk >= a.k)
                kk = 0;
            const int8_t* g;
            if (r < BM) {
                const uint32_t m = rows.lo + (uint32_t)r;
                g = a.a + (size_t)(m < rows.hi ? m : rows.hi - 1) * a.ld_a + kk;
            } else {
                const uint32_t n = n0 + (uint32_t)(r - BM);
                g = b + (size_t)(n < a.n ? n : a.n - 1) * a.ld_b + kk;
            }
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                             (__attribute__((address_space(3))) void*)&lds[buf][(i * 256 + wave * kWave) * 16],
                                             16, 0, 0);
        }
    };

    const int wm = (wave / 2) * 64, wn = (wave % 2) * 64;
    i32x16 acc[2][2] = {};
    if (stages > 0)
        load(0, 0);
    for (int st = 0; st < stages; ++st) {
        const int buf = st & 1;
        __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): this stage's loads of this wave
        __syncthreads();                      // ... of every wave; and the other buffer is free
        if (st + 1 < stages)
            load(st + 1, buf ^ 1);
        const int left = (int)a.k - st * kStep;
#pragma unroll
        for (int s = 0; s < kStep / 32; ++s) {
            i32x4 fa[2], fb[2];
            const int c = s * 2 + lane / 32;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int ra = wm + i * 32 + lane % 32, rb = wn + i * 32 + lane % 32;
                fa[i] = *reinterpret_cast<const i32x4*>(&lds[buf][(ra * 8 + (c ^ (ra & 7))) * 16]);
                fb[i] = *reinterpret_cast<const i32x4*>(&lds[buf][((BM + rb) * 8 + (c ^ (rb & 7))) * 16]);
            }
            if (left < kStep) {
                fa[0] = mask_bytes(fa[0], left - c * 16);
                fa[1] = mask_bytes(fa[1], left - c * 16);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
        }
    }

    // lane: token lane % 32, channels 8 (reg / 4) + 4 (lane / 32) + reg % 4
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t m = rows.lo + (uint32_t)(wm + i * 32 + lane % 32);
        if (m >= rows.hi)
            continue;
        const float sa = a.a_scales[m];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const uint32_t n = n0 + (uint32_t)(wn + j * 32 + 8 * (r / 4) + 4 * (lane / 32) + r % 4);
                if (n < a.n)
                    st_out<DT>(a, m, n, (float)acc[i][j][r] * sa * a.b_scales[(size_t)rows.expert * a.n + n]);
            }
    }
}

}  // namespace

hipError_t launch_quant_i8(const QuantI8Args& in, int dtype, hipStream_t s)
{
    QuantI8Args a = in;
    void* params[] = {&a};
    const bool tail = partial(a.k, dtype);
    const void* fn = dtype == 0 ? (tail ? (const void*)k_quant_i8<0, true> : (const void*)k_quant_i8<0, false>)
                                : (tail ? (const void*)k_quant_i8<1, true> : (const void*)k_quant_i8<1, false>);
    return launch_logged("k_quant_i8", fn, dim3((unsigned)a.rows), dim3(threads_for(vectors(a.k, dtype), 256)), params, s);
}

hipError_t launch_gemm_i8(const GemmI8Args& in, int out_dtype, hipStream_t s)
{
    GemmI8Args a = in;
    void* params[] = {&a};
    const size_t bm = 128, bn = 128;
    // experts: each may end in a partial tile, and so may the rows past them
    const size_t owners = (size_t)a.experts < a.rows ? (size_t)a.experts : a.rows;
    const size_t tm = a.offsets ? a.rows / bm + owners + 1 : (a.rows + bm - 1) / bm;
    const size_t grid = tm * ((a.n + bn - 1) / bn);
    return launch_logged("k_gemm_i8", out_dtype == 0 ? (const void*)k_gemm_i8<0> : (const void*)k_gemm_i8<1>,
                         dim3((unsigned)grid), dim3(256), params, s);
}

}  // namespace rx
