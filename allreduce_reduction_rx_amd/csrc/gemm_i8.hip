// gemm_i8.hip -- rows to 8-bit integers with a scale each, and the product of
// such matrices with a scale per token and channel, dense or grouped by
// expert (gfx950). Defined in rx.h.
#include <math.h>

#include "expert_tiles.hpp"

namespace rx {
namespace {

// A workgroup a row; up to NV vectors a thread stay in registers between the
// maximum and the codes, the rest of a longer row is read again.
template <int DT, bool TAIL, int NV>
__global__ __launch_bounds__(256) void k_quant_i8(QuantI8Args a)
{
    __shared__ uint32_t lds[4];
    const int tid = threadIdx.x, bd = blockDim.x;
    const size_t t = blockIdx.x;
    const int k = (int)a.k;
    const int nvec = (k + Elem<DT>::kVE - 1) / Elem<DT>::kVE;
    const void* row = static_cast<const char*>(a.x) + t * a.ld_x * Elem<DT>::kBytes;
    u32x4 x[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u)
        x[u] = ld_raw<DT, TAIL, true>(row, tid + u * bd, k);
#pragma unroll
    for (int u = 0; u < NV; ++u)
        x[u] = fixed<DT, TAIL>(x[u], tid + u * bd, k);
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < NV; ++u)
        m = umax(m, vec_absmax<DT>(x[u]));
    for (int v = tid + NV * bd; v < nvec; v += bd)
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
    uint32_t q[2];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        i8_codes<DT>(x[u], r, q);
        st_codes<DT, TAIL>(out, tid + u * bd, k, q);
    }
    for (int v = tid + NV * bd; v < nvec; v += bd) {
        i8_codes<DT>(ld_row<DT, TAIL>(row, v, k), r, q);
        st_codes<DT, TAIL>(out, v, k, q);
    }
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

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

// Results of 16 x 16 products: a lane holds row lane % 16 and channels
// 4 (lane / 16) + reg. Two neighbouring tiles of 16 channels are exchanged so
// that a lane stores eight channels at once.
template <int DT, int TM, int TN>
__device__ __forceinline__ void write_results(const GemmI8Args& a, const TileRows& rows, uint32_t row0, uint32_t col0,
                                              const i32x4 (*acc)[TN])
{
    const int lane = lane_id();
    float sa[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const uint32_t m = row0 + (uint32_t)(i * 16 + lane % 16);
        sa[i] = m < rows.hi ? a.a_scales[m] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < TN; j += 2) {
        // lane group g: tile j + g % 2, channels 8 (g / 2) + 0 .. 7
        const int g = lane / 16;
        const uint32_t n = col0 + (uint32_t)((j + g % 2) * 16 + g / 2 * 8);
        const float* bs = a.b_scales + (size_t)rows.expert * a.n + n;
        float sb[8];
        if (n + 8 <= a.n) {
            unpack<0>(ld16_any(bs), sb);
            unpack<0>(ld16_any(bs + 4), sb + 4);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sb[e] = n + e < a.n ? bs[e] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const uint32_t m = row0 + (uint32_t)(i * 16 + lane % 16);
            float o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                auto x = __builtin_amdgcn_permlane16_swap((uint32_t)acc[i][j][k], (uint32_t)acc[i][j + 1][k], false, false);
                o[k] = (float)(int)x[0] * sa[i] * sb[k];
                o[4 + k] = (float)(int)x[1] * sa[i] * sb[4 + k];
            }
            if (m < rows.hi && n < a.n)
                st_out8<DT>(a, m, n, o);
        }
    }
}

// BM x BN outputs, WM x WN waves. Stages of 128 bytes of k go from global
// memory to LDS directly (16 bytes a lane, LDS written in lane order), up to NBUF
// stages ahead. Chunk c of row r sits where the sixteen rows that one pass
// of a 16-byte read touches lie in different banks; the load picks its global
// chunk to match. Rows past the end read the last row, chunks past k read
// chunk 0 and are masked out of `a` in the last stage. The fragments of the
// next 64 bytes of k are read while this one's products run, so a stage's last
// read is over half a stage before its end and its buffer is filled again a
// whole stage before it is needed.
//
// What bounds it. At 8192^3 in 256 x 256 tiles, the same operands over and over,
// the clock falls from 2.4 to 1.9 GHz with the matrix cores busy 68% of the
// cycles: power (393 to 447 us from card to card, 2.80 to 2.46 POP/s; a large library
// product reaches 2.54 to 2.44). With operands that are in no cache it stays at
// 2.2 GHz, busy 53% (457 us): the start of each of four rounds waits for memory
// too. What saves instructions and bytes saved time: products of 16 x 16 x 64
// move half the accumulators a multiply that 32 x 32 x 32 do (494 against 510
// us before the earlier refill), 128-byte stages half the requests of 64-byte
// ones, eight waves of 64 x 128 keep all fragments in registers.
template <int DT, int BM, int BN, int WM, int WN, int NBUF>
__global__ __launch_bounds__(WM * WN * kWave, 1) void k_gemm_i8(GemmI8Args a)
{
    constexpr int kThreads = WM * WN * kWave, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int BK = 128, kChunks = BK / 16, kSteps = BK / 64, kStage = (BM + BN) * BK;
    constexpr int NL = kStage / 16 / kThreads;            // loads of a thread and stage
    constexpr int kRowsALoad = kThreads / kChunks;
    static_assert(kStage % (16 * kThreads) == 0 && kRowsALoad % 16 == 0 && (NBUF - 1) * NL < 64 && BM % kRowsALoad == 0, "");
    __shared__ __align__(16) int8_t lds[NBUF][kStage];
    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
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
    const int8_t* b = a.b + (size_t)rows.expert * a.stride_b;
    const int stages = (int)((a.k + BK - 1) / BK);

    // where chunk c of row r sits in its row
    auto place = [](int r, int c) { return c ^ ((r >> 1) & 7); };
    const int lr = tid / kChunks, lc = place(lr, tid % kChunks);   // kRowsALoad is a multiple of 16
    uint32_t from[NL];   // below 2^31: 256 rows of a stride below 2^23
    const int8_t* abase = a.a + (size_t)rows.lo * a.ld_a;
    const int8_t* bbase = b + (size_t)n0 * a.ld_b;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const uint32_t r = (uint32_t)(i * kRowsALoad + lr);
        if (i * kRowsALoad < BM) {
            const uint32_t most = rows.hi - 1 - rows.lo;
            from[i] = (r < most ? r : most) * (uint32_t)a.ld_a;
        } else {
            const uint32_t most = a.n - 1 - n0;
            from[i] = (r - BM < most ? r - BM : most) * (uint32_t)a.ld_b;
        }
    }
    // load i of a stage
    auto load = [&](int st, int buf, int i) {
        uint32_t kk = (uint32_t)(st * BK + lc * 16);
        if (kk >= a.k)
            kk = 0;
        const int8_t* g = (i * kRowsALoad < BM ? abase : bbase) + (from[i] + kk);
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                         (__attribute__((address_space(3))) void*)&lds[buf][(i * kThreads + wave * kWave) * 16],
                                         16, 0, 0);
    };

    const int wm = (wave / WN) * TM * 16, wn = (wave % WN) * TN * 16;
    const int ar = wm + lane % 16, br = BM + wn + lane % 16;
    i32x4 acc[TM][TN] = {};
    i32x4 fa[2][TM], fb[2][TN];
    // fragment f of step s: fa[0], the fbs, then the other fas
    auto read = [&](int buf, int s, int set, int f) {
        const int c = s * 4 + lane / 16;
        if (f >= 1 && f <= TN)
            fb[set][f - 1] = *reinterpret_cast<const i32x4*>(&lds[buf][br * BK + place(br, c) * 16 + (f - 1) * 16 * BK]);
        else {
            const int i = f ? f - TN : 0;
            fa[set][i] = *reinterpret_cast<const i32x4*>(&lds[buf][ar * BK + place(ar, c) * 16 + i * 16 * BK]);
        }
    };
    auto multiply = [&](int set, int m) {
        acc[m / TN][m % TN] =
            __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[set][m % TN], fa[set][m / TN], acc[m / TN][m % TN], 0, 0, 0);
    };
    auto open_stage = [&] {
        wait_lds();
        wait_loads<(NBUF - 2) * NL>();
        order();
        __builtin_amdgcn_s_barrier();
        order();
    };

    if (stages > 0 && rows.lo + (uint32_t)wm >= rows.hi) {
        // no rows for this wave: it loads its share and keeps the barriers
        for (int st = -1; st < stages - 1; ++st) {
            const int from_st = st < 0 ? 0 : st + NBUF, n_st = st < 0 ? NBUF : 1;
            if (st >= 0)
                open_stage();
            for (int f = 0; f < n_st; ++f)
#pragma unroll
                for (int i = 0; i < NL; ++i)
                    load(from_st + f < stages ? from_st + f : stages - 1, st < 0 ? f : st % NBUF, i);
            if (st < 0) {
                wait_loads<(NBUF - 1) * NL>();
                order();
                __builtin_amdgcn_s_barrier();
                order();
            }
        }
        wait_loads<0>();   // nothing writes LDS after the wave's end
        return;
    }
    if (stages > 0) {
        // a stage past the last is the last again, read by nobody: no branch
        // and one wait for all
        auto stage = [&](int st) { return st < stages ? st : stages - 1; };
#pragma unroll
        for (int st = 0; st < NBUF; ++st) {
#pragma unroll
            for (int i = 0; i < NL; ++i)
                load(stage(st), st, i);
        }
        wait_loads<(NBUF - 1) * NL>();
        order();
        __builtin_amdgcn_s_barrier();
        order();
#pragma unroll
        for (int f = 0; f < TM + TN; ++f)
            read(0, 0, 0, f);
        int buf = 0;
        for (int st = 0; st < stages - 1; ++st) {
            const int next = buf + 1 == NBUF ? 0 : buf + 1;
            // after each product its share of the next step's reads, in the
            // last step of the loads too: the matrix pipe waits for neither
            unrolled<kSteps * TM * TN>([&](auto at) {
                constexpr int s = at() / (TM * TN), m = at() % (TM * TN), F = TM + TN;
                constexpr bool last = s == kSteps - 1;
                constexpr int first = last ? 2 : 0, items = F + (last ? NL : 0), slots = TM * TN - first;
                multiply(s & 1, m);
                if constexpr (last && m == 1)
                    // every wave has read its last fragments of this stage, so
                    // its buffer is free; the next stage has arrived
                    open_stage();
                unrolled<items>([&](auto item) {
                    constexpr int i = item();
                    if constexpr (i * slots / items + first == m) {
                        if constexpr (i < F)
                            read(last ? next : buf, last ? 0 : s + 1, (s + 1) & 1, i);
                        else
                            load(stage(st + NBUF), buf, i - F);
                    }
                });
                __builtin_amdgcn_sched_barrier(0);
            });
            buf = next;
        }
        const int left = (int)a.k - (stages - 1) * BK;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            if (left < BK) {
                const int nb = left - (s * 4 + lane / 16) * 16;
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    fa[s & 1][i] = mask_bytes(fa[s & 1][i], nb);
            }
            if (s + 1 < kSteps)
#pragma unroll
                for (int f = 0; f < TM + TN; ++f)
                    read(buf, s + 1, (s + 1) & 1, f);
#pragma unroll
            for (int m = 0; m < TM * TN; ++m)
                multiply(s & 1, m);
        }
        wait_loads<0>();   // nothing writes LDS after the wave's end
    }
    write_results<DT, TM, TN>(a, rows, rows.lo + (uint32_t)wm, n0 + (uint32_t)wn, acc);
}

// Few rows: 16 MT rows x 16 NT channels a workgroup, and the stages of k
// dealt to its waves. Each wave fills a ring of NBUF stages of its own, so
// nothing waits at a barrier until the waves' exact sums meet in LDS, and a
// CU keeps W (NBUF - 1) stages in flight: such products are bound by the
// bytes of b.
template <int DT, int MT, int NT, int W, int NBUF>
__global__ __launch_bounds__(W * kWave) void k_gemm_i8_split(GemmI8Args a)
{
    constexpr int BM = 16 * MT, BN = 16 * NT, BK = 128, NL = (BM + BN) / 8, kStage = (BM + BN) * BK;
    static_assert((NBUF - 1) * NL < 64 && NBUF >= 2 && NBUF <= 4, "");
    __shared__ __align__(16) int8_t ring[W][NBUF][kStage];
    static_assert(sizeof(ring) >= sizeof(i32x4) * W * MT * NT * kWave, "");
    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
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
    const int8_t* abase = a.a + (size_t)rows.lo * a.ld_a;
    const int8_t* bbase = a.b + (size_t)rows.expert * a.stride_b + (size_t)n0 * a.ld_b;
    uint32_t from[NL];   // below 2^31, as above
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const uint32_t r = (uint32_t)(i * 8 + lane / 8);
        if (i * 8 < BM) {
            const uint32_t most = rows.hi - 1 - rows.lo;
            from[i] = (r < most ? r : most) * (uint32_t)a.ld_a;
        } else {
            const uint32_t most = a.n - 1 - n0;
            from[i] = (r - BM < most ? r - BM : most) * (uint32_t)a.ld_b;
        }
    }
    auto place = [](int r, int c) { return c ^ ((r >> 1) & 7); };
    const int stages = (int)((a.k + BK - 1) / BK), mine = stages > wave ? (stages - wave + W - 1) / W : 0;
    auto load = [&](int i, int buf) {   // this wave's stage i
        const uint32_t k0 = (uint32_t)(wave + i * W) * BK;
        uint32_t kk[2];   // of the even and the odd groups of eight rows
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            kk[e] = k0 + (uint32_t)place(e * 8 + lane / 8, lane % 8) * 16;
            if (kk[e] >= a.k)
                kk[e] = 0;
        }
#pragma unroll
        for (int l = 0; l < NL; ++l)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)((l * 8 < BM ? abase : bbase) + (from[l] + kk[l & 1])),
                                             (__attribute__((address_space(3))) void*)&ring[wave][buf][l * 1024], 16, 0, 0);
    };

    i32x4 acc[MT][NT] = {};
    for (int i = 0; i < NBUF && i < mine; ++i)
        load(i, i);
    int buf = 0;
    for (int i = 0; i < mine; ++i) {
        const int after = mine - 1 - i;   // stages still to come
        if (NBUF > 3 && after >= 3)
            wait_loads<(NBUF > 3 ? 3 : 0) * NL>();
        else if (NBUF > 2 && after >= 2)
            wait_loads<(NBUF > 2 ? 2 : 0) * NL>();
        else if (after >= 1)
            wait_loads<NL>();
        else
            wait_loads<0>();
        order();
        i32x4 fa[2][MT], fb[2][NT];
        const int8_t* p = ring[wave][buf];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int c = s * 4 + lane / 16;
#pragma unroll
            for (int m = 0; m < MT; ++m)
                fa[s][m] = *reinterpret_cast<const i32x4*>(p + (m * 16 + lane % 16) * BK + place(lane % 16, c) * 16);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                fb[s][n] = *reinterpret_cast<const i32x4*>(p + (BM + n * 16 + lane % 16) * BK + place(lane % 16, c) * 16);
        }
        order();
        wait_lds();   // read before it is written again
        order();
        if (i + NBUF < mine)
            load(i + NBUF, buf);
        buf = buf + 1 == NBUF ? 0 : buf + 1;
        const int left = (int)a.k - (wave + i * W) * BK;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (left < BK)
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    fa[s][m] = mask_bytes(fa[s][m], left - (s * 4 + lane / 16) * 16);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[m][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[s][n], fa[s][m], acc[m][n], 0, 0, 0);
        }
    }
    __syncthreads();   // the rings are free
    i32x4* part = reinterpret_cast<i32x4*>(&ring[0][0][0]);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            part[((wave * MT + m) * NT + n) * kWave + lane] = acc[m][n];
    __syncthreads();
    // a wave joins the sums of 16 x 16 results: a lane four channels of a row
    for (int t = wave; t < MT * NT; t += W) {
        i32x4 sum = part[t * kWave + lane];
#pragma unroll
        for (int w = 1; w < W; ++w)
            sum += part[(w * MT * NT + t) * kWave + lane];
        const uint32_t m = rows.lo + (uint32_t)(t / NT * 16 + lane % 16), n = n0 + (uint32_t)(t % NT * 16 + lane / 16 * 4);
        if (m >= rows.hi)
            continue;
        const float sa = a.a_scales[m];
        char* p = static_cast<char*>(a.out) + ((size_t)m * a.ld_out + n) * Elem<DT>::kBytes;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < a.n) {
                const float v = (float)sum[e] * sa * a.b_scales[(size_t)rows.expert * a.n + n + e];
                if constexpr (DT == 0)
                    reinterpret_cast<float*>(p)[e] = v;
                else
                    reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)pack_bf16(v, 0.0f);
            }
    }
}

}  // namespace

template <int NV>
const void* quant_fn(int dtype, bool tail)
{
    if (dtype == 0)
        return tail ? (const void*)k_quant_i8<0, true, NV> : (const void*)k_quant_i8<0, false, NV>;
    return tail ? (const void*)k_quant_i8<1, true, NV> : (const void*)k_quant_i8<1, false, NV>;
}

hipError_t launch_quant_i8(const QuantI8Args& in, int dtype, hipStream_t s)
{
    QuantI8Args a = in;
    void* params[] = {&a};
    const bool tail = partial(a.k, dtype);
    const size_t nvec = vectors(a.k, dtype);
    const unsigned wg = threads_for(nvec, 256);
    const size_t nv = (nvec + wg - 1) / wg;
    const void* fn = nv <= 1 ? quant_fn<1>(dtype, tail) : nv <= 4 ? quant_fn<4>(dtype, tail) : quant_fn<8>(dtype, tail);
    return launch_logged("k_quant_i8", fn, dim3((unsigned)a.rows), dim3(wg), params, s);
}

hipError_t launch_grid(GemmI8Args& a, const void* fn, const char* name, size_t bm, size_t bn, unsigned threads, hipStream_t s)
{
    void* params[] = {&a};
    // whole rounds of the XCDs for the tiles with an expert and for those without
    const size_t grid = (row_tiles(a, bm) * ((a.n + bn - 1) / bn) + 2 * kXcds) / kXcds * kXcds;
    return launch_logged(name, fn, dim3((unsigned)grid), dim3(threads), params, s);
}

template <int BM, int BN, int WM, int WN, int NBUF>
hipError_t launch_tiles(GemmI8Args& a, int out_dtype, hipStream_t s)
{
    const void* fn = out_dtype == 0 ? (const void*)k_gemm_i8<0, BM, BN, WM, WN, NBUF> : (const void*)k_gemm_i8<1, BM, BN, WM, WN, NBUF>;
    return launch_grid(a, fn, "k_gemm_i8", BM, BN, WM * WN * kWave, s);
}

template <int MT, int NT, int W, int NBUF>
hipError_t launch_split(GemmI8Args& a, int out_dtype, hipStream_t s)
{
    const void* fn = out_dtype == 0 ? (const void*)k_gemm_i8_split<0, MT, NT, W, NBUF> : (const void*)k_gemm_i8_split<1, MT, NT, W, NBUF>;
    return launch_grid(a, fn, "k_gemm_i8_split", 16 * MT, 16 * NT, W * kWave, s);
}

// Estimated time, in microseconds for every 128 bytes of k. `us` is what a
// round of a kind takes with the GPU full, measured: 1.71 for 256 x 256 (8192^3,
// 439 us in four rounds), 1.05 for 128 x 256 (2048 x 4096 x 4096, 34 us), 0.65
// for 128 x 128 with eight waves (512 x 8192 x 8192, 42 us), 1.14 for two of 128 x
// 128 with four waves a CU (8192^3, 586 us), 0.53 for two of 64 x 64 (512 x 8192
// x 8192, 68 us), 0.36 for two of 32 x 32 with split k (64 x 8192 x 8192, 23 us).
//
// A call pays whole rounds where a CU has one workgroup at a time (one tile
// more than 256 cost 44 us instead of 27 us in a call over 24 experts); with
// two, the last round's run faster alone. With experts the number of tiles
// is known to about half a tile each, half a round in the mean.
//
// Where each would go wrong: 32 x 8192 x 8192 takes 14 us split and 57 us in
// 256 x 256; 32116 rows of 32 experts x 4096 x 4096 take 571 us in 256 x 256, 602 in
// 128 x 256, 732 in 128 x 128, 1048 in 64 x 64 and 1851 split; 2007 rows of 24
// experts x 2100 x 2056 take 32 us in two of 128 x 128, 44 in 128 x 256, 37 in 256 x 256.
double estimate(const GemmI8Args& a, double bm, double bn, double per_cu, double us)
{
    double tm = (double)((a.rows + (size_t)bm - 1) / (size_t)bm);
    if (a.offsets) {
        const double owners = (double)a.experts < a.rows ? (double)a.experts : a.rows;
        tm = a.rows / bm + 0.5 * owners;
        tm = tm < owners ? owners : tm;
    }
    const double tn = (double)((a.n + (size_t)bn - 1) / (size_t)bn), t = tm * tn / (per_cu * device_cu_count());
    if (((double)row_tiles(a, (size_t)bm) * tn + 16.0) * 512.0 >= 4294967296.0)
        return 1e300;   // threads of one launch
    const double whole = ceil(t);
    if (t <= 1.0)
        return us;
    if (per_cu > 1.0)
        return us * (t + 0.25 < whole ? t + 0.25 : whole);
    return us * (a.offsets ? t + 0.5 : whole);
}

hipError_t launch_gemm_i8(const GemmI8Args& in, int out_dtype, hipStream_t s)
{
    GemmI8Args a = in;
    const double cost[] = {estimate(a, 256, 256, 1, 1.71), estimate(a, 128, 256, 1, 1.05), estimate(a, 128, 128, 1, 0.65),
                           estimate(a, 128, 128, 2, 1.14), estimate(a, 64, 64, 2, 0.53), estimate(a, 32, 32, 2, 0.36)};
    int best = 0;
    for (int i = 1; i < 6; ++i)
        if (cost[i] < cost[best])
            best = i;
    switch (best) {
    case 0: return launch_tiles<256, 256, 4, 2, 2>(a, out_dtype, s);
    case 1: return launch_tiles<128, 256, 2, 4, 3>(a, out_dtype, s);
    case 2: return launch_tiles<128, 128, 2, 4, 4>(a, out_dtype, s);
    case 3: return launch_tiles<128, 128, 2, 2, 2>(a, out_dtype, s);
    case 4: return launch_tiles<64, 64, 2, 2, 4>(a, out_dtype, s);
    default: return launch_split<2, 2, 4, 2>(a, out_dtype, s);
    }
}

}  // namespace rx
