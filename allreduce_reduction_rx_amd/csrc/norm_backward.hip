// norm_backward.hip -- the gradient of the sum over the ranks fused with the
// norms, the gate and the residual around a block (gfx950). Defined in rx.h.
//
// The gradient. A workgroup takes a range of rows (a part), R teams of
// WG / R threads a row each at a time, and keeps the parameters' sums of its
// part; k_norm_params adds the parts in their order.
//
// With c = g w_post, e = d_h + q a and dH = e - h m1, m1 = q^3 S1 / H,
// S1 = sum a h, the second mean is sum(c dH y) / H = (S2 - m1 S3) / H with
// S2 = sum c e y, S3 = sum c h y: the three sums cross the team together,
// and an element costs about 30 instructions. Both d_gate and d_w_post come
// from one sum over the rows of a gate row, T = sum dH y p: d_gate = w_post T,
// and d_w_post gains g T. Operands that are absent are neutral values (ones,
// zeros), so the arithmetic has no branches.
//
// The next row's loads go out as soon as this row's are unpacked, before the
// sums, the results and the stores of this row: 80 KiB in flight a CU. HBM
// bound: 16384 x 8192 BF16 over two sources takes 370 us for 1.88 GB read and
// written (5.1 TB/s; large copies reach 5.0 to 5.8).
//
// MULTI: the part may see several gate rows. A gate row whose rows all lie in
// the part is written at once; one that crosses the part's start goes to
// slot 0 of the part's two, one that only crosses its end to slot 1.
// ACC: the parameters' sums stay in LDS instead of registers: rows of 1025 to
// 1536 vectors in BF16 (three vectors a thread; 4096 x 10240, forward and
// backward: 296 us, 344 with 1024 threads), and all rows of 1537 to 2048, where
// 1024 threads leave 128 registers a thread and nothing is loaded ahead (4096 x
// 16384 BF16: 432 us, against 717 us with four vectors a thread loaded ahead and
// 807 us with k_norm_backward_long, which takes the rows above; 457 with inputs
// that are in no cache, 323 of them this direction's). Both are far from the memory:
// 4096 rows of FP32 take 224 us at 8192 (1024 threads) and 640 at 16384 (long).
#include "norm_common.hpp"

namespace rx {
namespace {

// c += x, kept in registers or, four at a time `stride` apart, in LDS.
template <bool ACC, int N>
__device__ __forceinline__ void add_to(float* c, u32x4* lds, int stride, const float* x)
{
    if constexpr (ACC) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            u32x4 v = lds[i * stride];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = __builtin_bit_cast(uint32_t, bits_f32(v[k]) + x[4 * i + k]);
            lds[i * stride] = v;
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
            c[k] += x[k];
    }
}

// x = c, c = 0.
template <bool ACC, int N>
__device__ __forceinline__ void take(float* c, u32x4* lds, int stride, float* x)
{
    if constexpr (ACC) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const u32x4 v = lds[i * stride];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                x[4 * i + k] = bits_f32(v[k]);
            lds[i * stride] = u32x4{0, 0, 0, 0};
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            x[k] = c[k];
            c[k] = 0.0f;
        }
    }
}

// x summed over the teams in their order, right in team 0.
template <int R, int W, int N>
__device__ __forceinline__ void join_teams(float* x, int team, int tid, float* lds)
{
    if constexpr (R > 1) {
        __syncthreads();   // the previous use of lds is over
#pragma unroll
        for (int k = 0; k < N; ++k)
            lds[(team * N + k) * W + tid] = x[k];
        __syncthreads();
        if (team == 0)
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int r = 1; r < R; ++r)
                    x[k] += lds[(r * N + k) * W + tid];
    }
}

// Keeps x a value of this iteration: what is computed from it is computed
// here again instead of being held in registers over the whole loop.
__device__ __forceinline__ u32x4 held(u32x4 x)
{
    asm("" : "+v"(x));
    return x;
}

__device__ __forceinline__ u32x4 ones(int dt)
{
    const uint32_t o = dt ? 0x3F803F80u : 0x3F800000u;
    return u32x4{o, o, o, o};
}

// N floats of a row of sums from column c on, and back.
template <int N>
__device__ __forceinline__ void st_sums(float* row, uint32_t c, uint32_t hidden, const float* x)
{
    if (c + N <= hidden) {
#pragma unroll
        for (int k = 0; k < N; k += 4)
            st16_any(row + c + k, pack<0>(x + k));
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (c + k < hidden)
                row[c + k] = x[k];
    }
}
template <int N>
__device__ __forceinline__ void ld_sums(const float* row, uint32_t c, uint32_t hidden, float* x)
{
#pragma unroll
    for (int k = 0; k < N; k += 4)
        if (c + N <= hidden)
            unpack<0>(ld16_any(row + c + k), x + k);
        else
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[k + i] = c + k + i < hidden ? row[c + k + i] : 0.0f;
}

// One vector of a row up to the three sums: h, e, and d_w_pre's term.
template <int DT, int VE>
__device__ __forceinline__ void row_sums(const float* y, u32x4 res, u32x4 dhv, u32x4 dzv, u32x4 wpost, u32x4 wpre,
                                         u32x4 gate, float p, float q, float rs, float* h, float* e, float* pre, float* s)
{
    float w1[VE], w2[VE], g[VE], f[VE], dz[VE], dh[VE];
    unpack<DT>(wpost, w1);
    unpack<DT>(wpre, w2);
    unpack<DT>(gate, g);
    unpack<DT>(res, f);
    unpack<DT>(dzv, dz);
    unpack<DT>(dhv, dh);
#pragma unroll
    for (int k = 0; k < VE; ++k) {
        const float cy = g[k] * w1[k] * y[k];
        h[k] = __builtin_fmaf(cy, p, rs * f[k]);
        const float zh = dz[k] * h[k];
        pre[k] = zh * q;
        e[k] = __builtin_fmaf(q, dz[k] * w2[k], dh[k]);
        s[0] = __builtin_fmaf(zh, w2[k], s[0]);
        s[1] = __builtin_fmaf(cy, e[k], s[1]);
        s[2] = __builtin_fmaf(cy, h[k], s[2]);
    }
}

// ... and from the sums on: d_residual, d_src, and T's term.
template <int DT, int VE>
__device__ __forceinline__ void row_results(const float* y, const float* h, const float* e, u32x4 wpost, u32x4 gate,
                                            float p, float m1, float m2, float rs, float* o1, float* o2, float* t)
{
    float w1[VE], g[VE];
    unpack<DT>(wpost, w1);
    unpack<DT>(gate, g);
#pragma unroll
    for (int k = 0; k < VE; ++k) {
        const float dH = __builtin_fmaf(-m1, h[k], e[k]);
        o1[k] = rs * dH;
        t[k] = dH * (y[k] * p);
        o2[k] = p * __builtin_fmaf(-m2, y[k], g[k] * w1[k] * dH);
    }
}

// The two means, from the three sums, multiplied outwards from the sum: S1 / H
// is at most rms(a) / q, so every step lies between it and the result. q^3
// by itself would leave FP32's range for rows of 1e13 or more, and be infinite
// for a row of zeros with eps below 2e-26, whose mean is 0.
__device__ __forceinline__ void row_means(const NormBwdArgs& a, const float* s, float p, float q, float& m1, float& m2)
{
    m1 = s[0] * a.inv_hidden * q * q * q;
    m2 = a.w_post ? (s[1] - m1 * s[2]) * a.inv_hidden * p * p : 0.0f;
}

// Where the sum of gate row grp goes from this part.
__device__ __forceinline__ float* gate_target(const NormBwdArgs& a, size_t grp, size_t r0, size_t r1)
{
    const size_t g0 = grp * a.gate_rows;
    const size_t g1 = g0 + a.gate_rows < a.rows ? g0 + a.gate_rows : a.rows;
    if (a.d_gate && g0 >= r0 && g1 <= r1)
        return a.d_gate + grp * a.hidden;
    return a.part_gate + (blockIdx.x * 2 + (g0 < r0 ? 0 : 1)) * a.hidden;
}

template <int DT, bool TAIL, int NV, int WG, int R, bool MULTI, bool ACC>
__global__ __launch_bounds__(WG, WG > 512 ? 4 : 2) void k_norm_backward(NormBwdArgs a)
{
    constexpr int VE = Elem<DT>::kVE, EB = Elem<DT>::kBytes, W = WG / R, E = NV * VE;
    constexpr int PS = ACC ? 2 : 4;   // sources loaded together with the rest
    constexpr bool kAhead = WG <= 512;
    static_assert(R == 1 || W == kWave, "teams of several waves share no barriers");
    __shared__ float sums[2 * 16 * 3];
    __shared__ __align__(16) float dyn[ACC ? 2 * W * E : R > 1 ? R * W * VE : 4];
    int turn = 0;
    const int hidden = (int)a.hidden;
    const int team = R == 1 ? 0 : (int)__builtin_amdgcn_readfirstlane(threadIdx.x / W);
    const int tid = (int)threadIdx.x - team * W;
    const size_t r0 = blockIdx.x * a.part_rows;
    const size_t r1 = r0 + a.part_rows < a.rows ? r0 + a.part_rows : a.rows;

    float acc_t[E] = {}, acc_pre[E] = {};
    // where registers are short the weights and the gate wait in LDS (4096 x
    // 5120 FP32 with a gate for each 100 rows, both directions: 266 -> 206 us)
    constexpr bool kWeightsInLds = !ACC && (NV == 3 || (MULTI && NV == 2 && DT == 1));
    __shared__ u32x4 wlds[kWeightsInLds ? 3 : 1][kWeightsInLds ? NV : 1][kWeightsInLds ? WG : 1];
    u32x4 wreg[3][NV];
    auto keep = [&](int which, int u, u32x4 x) {   // 0: w_post, 1: w_pre, 2: the gate
        if constexpr (kWeightsInLds)
            wlds[which][u][threadIdx.x] = x;
        else
            wreg[which][u] = x;
    };
    auto kept = [&](int which, int u) {
        if constexpr (kWeightsInLds)
            return wlds[which][u][threadIdx.x];
        else
            return held(wreg[which][u]);
    };
    u32x4* lt = reinterpret_cast<u32x4*>(dyn) + tid;
    u32x4* lp = lt + (size_t)W * (E / 4);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int v = tid + u * W;
        keep(0, u, a.w_post ? ld_row<DT, TAIL>(a.w_post, v, hidden) : ones(DT));
        keep(1, u, a.w_pre ? ld_row<DT, TAIL>(a.w_pre, v, hidden) : ones(DT));
        keep(2, u, ones(DT));
    }
    if constexpr (ACC)
#pragma unroll
        for (int i = 0; i < E / 4; ++i)
            lt[i * W] = lp[i * W] = u32x4{0, 0, 0, 0};

    u32x4 src[PS][NV], res[NV], dhv[NV], dzv[NV];
    float np = 1.0f, nq = 0.0f;
    auto load = [&](size_t t) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int v = tid + u * W;
            const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
            for (int r = 0; r < PS; ++r)
                if (r < a.nsrc)
                    src[r][u] = ld_raw<DT, TAIL, true>(static_cast<const char*>(a.src[r]) + t * a.ld_src * EB, v, hidden);
            res[u] = a.residual ? ld_raw<DT, TAIL, true>(static_cast<const char*>(a.residual) + t * a.ld_residual * EB, v, hidden) : zero;
            dhv[u] = a.d_h ? ld_raw<DT, TAIL, true>(static_cast<const char*>(a.d_h) + t * a.ld_d_h * EB, v, hidden) : zero;
            dzv[u] = a.d_z ? ld_raw<DT, TAIL, true>(static_cast<const char*>(a.d_z) + t * a.ld_d_z * EB, v, hidden) : zero;
        }
        if (a.w_post)
            np = a.rstd_post[t];
        if (a.d_z)
            nq = a.rstd_pre[t];
    };

    // one team: a part's rows follow each other; several: each gate row's
    // first rows are loaded where they are needed
    constexpr bool kRun = kAhead && R == 1;
    if constexpr (kRun)
        load(r0);
    size_t have = ~(size_t)0, grp = r0 / a.gate_rows;
    for (size_t s0 = r0; s0 < r1; ++grp) {
        const size_t ge = (grp + 1) * a.gate_rows;
        const size_t s1 = ge < r1 ? ge : r1;
        if (a.gate)
#pragma unroll
            for (int u = 0; u < NV; ++u)
                keep(2, u, ld_row<DT, TAIL>(static_cast<const char*>(a.gate) + grp * a.hidden * EB, tid + u * W, hidden));
        for (size_t t = s0 + team; t < s1; t += R) {
            if (!kRun && have != t)
                load(t);
            const float p = np, q = nq;
            float y[NV][VE], h[NV][VE], e[NV][VE], s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                unpack<DT>(fixed<DT, TAIL>(src[0][u], tid + u * W, hidden), y[u]);
#pragma unroll
                for (int r = 1; r < PS; ++r)
                    if (r < a.nsrc) {
                        float f[VE];
                        unpack<DT>(fixed<DT, TAIL>(src[r][u], tid + u * W, hidden), f);
#pragma unroll
                        for (int k = 0; k < VE; ++k)
                            y[u][k] += f[k];
                    }
            }
            int r = PS;
            for (; r + 2 <= a.nsrc; r += 2)
                fold_batch<DT, TAIL, NV, 2, false>(a.src, r, t * a.ld_src * EB, hidden, tid, W, y);
            if (r < a.nsrc)
                fold_batch<DT, TAIL, NV, 1, false>(a.src, r, t * a.ld_src * EB, hidden, tid, W, y);
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                float pre[VE];
                auto whole = [&](u32x4 x) { return fixed<DT, TAIL>(x, tid + u * W, hidden); };
                row_sums<DT, VE>(y[u], whole(res[u]), whole(dhv[u]), whole(dzv[u]), kept(0, u), kept(1, u), kept(2, u), p, q,
                                 a.residual_scale, h[u], e[u], pre, s);
                add_to<ACC, VE>(acc_pre + u * VE, lp + u * (VE / 4) * W, W, pre);
            }
            const size_t next = t + R < s1 ? t + R : R == 1 ? s1 : r1;
            if (kAhead && next < r1) {
                load(next);
                have = next;
            }
            block_sums<3, W / kWave>(s, sums, turn);
            float m1, m2;
            row_means(a, s, p, q, m1, m2);
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                float o1[VE], o2[VE], tt[VE];
                row_results<DT, VE>(y[u], h[u], e[u], kept(0, u), kept(2, u), p, m1, m2, a.residual_scale, o1, o2, tt);
                add_to<ACC, VE>(acc_t + u * VE, lt + u * (VE / 4) * W, W, tt);
                const int v = tid + u * W;
                if (a.d_residual)
                    st_row<DT, TAIL, true>(static_cast<char*>(a.d_residual) + t * a.ld_d_residual * EB, v, hidden, pack<DT>(o1));
                st_row<DT, TAIL, true>(static_cast<char*>(a.d_src) + t * a.ld_d_src * EB, v, hidden, pack<DT>(o2));
            }
        }
        if constexpr (MULTI) {
            // this gate row's rows of the part are done
            float* to = gate_target(a, grp, r0, r1);
            float* post = a.part_post + blockIdx.x * a.hidden;
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                float w1[VE], g[VE], tv[VE];
                unpack<DT>(kept(0, u), w1);
                unpack<DT>(kept(2, u), g);
                take<ACC, VE>(acc_t + u * VE, lt + u * (VE / 4) * W, W, tv);
                join_teams<R, W, VE>(tv, team, tid, dyn);
                const uint32_t c = (uint32_t)((tid + u * W) * VE);
                if (team == 0 && c < (uint32_t)hidden) {
                    float sum[VE];
                    if (s0 > r0)
                        ld_sums<VE>(post, c, hidden, sum);
#pragma unroll
                    for (int k = 0; k < VE; ++k) {
                        sum[k] = s0 == r0 ? g[k] * tv[k] : sum[k] + g[k] * tv[k];
                        tv[k] *= w1[k];
                    }
                    st_sums<VE>(post, c, hidden, sum);
                    if (a.d_gate)
                        st_sums<VE>(to, c, hidden, tv);
                }
                __builtin_amdgcn_sched_barrier(0);   // one vector at a time: registers
            }
        }
        s0 = s1;
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float tv[VE], pre[VE];
        if constexpr (!MULTI) {
            take<ACC, VE>(acc_t + u * VE, lt + u * (VE / 4) * W, W, tv);
            join_teams<R, W, VE>(tv, team, tid, dyn);
        }
        take<ACC, VE>(acc_pre + u * VE, lp + u * (VE / 4) * W, W, pre);
        join_teams<R, W, VE>(pre, team, tid, dyn);
        const uint32_t c = (uint32_t)((tid + u * W) * VE);
        if (team == 0 && c < (uint32_t)hidden) {
            if constexpr (!MULTI)
                st_sums<VE>(a.part_post + blockIdx.x * a.hidden, c, hidden, tv);
            st_sums<VE>(a.part_pre + blockIdx.x * a.hidden, c, hidden, pre);
        }
    }
}

// Rows too long for the registers: the operands are read twice, the second
// time from the caches, and the parameters' sums are kept in the workspace
// itself (a thread adds to its own columns).
template <int DT, bool TAIL, bool MULTI>
__global__ __launch_bounds__(1024) void k_norm_backward_long(NormBwdArgs a)
{
    constexpr int VE = Elem<DT>::kVE, EB = Elem<DT>::kBytes;
    __shared__ float sums[2 * 16 * 3];
    int turn = 0;
    const int hidden = (int)a.hidden, nvec = (hidden + VE - 1) / VE;
    const size_t r0 = blockIdx.x * a.part_rows;
    const size_t r1 = r0 + a.part_rows < a.rows ? r0 + a.part_rows : a.rows;
    float* part_pre = a.part_pre + blockIdx.x * a.hidden;
    float* part_post = a.part_post + blockIdx.x * a.hidden;
    size_t grp = r0 / a.gate_rows;
    for (size_t s0 = r0; s0 < r1; ++grp) {
        const size_t ge = (grp + 1) * a.gate_rows;
        const size_t s1 = ge < r1 ? ge : r1;
        float* to = MULTI ? gate_target(a, grp, r0, r1) : part_post;
        const char* grow = a.gate ? static_cast<const char*>(a.gate) + grp * a.hidden * EB : nullptr;
        for (size_t t = s0; t < s1; ++t) {
            const float p = a.w_post ? a.rstd_post[t] : 1.0f, q = a.d_z ? a.rstd_pre[t] : 0.0f;
            float s[3] = {0.0f, 0.0f, 0.0f}, m1 = 0.0f, m2 = 0.0f;
#pragma unroll
            for (int pass = 0; pass < 2; ++pass) {
                for (int v = (int)threadIdx.x; v < nvec; v += 1024) {
                    const u32x4 zero = {0, 0, 0, 0};
                    auto row = [&](const void* base, size_t ld) {
                        return base ? ld_row<DT, TAIL>(static_cast<const char*>(base) + t * ld * EB, v, hidden) : zero;
                    };
                    const u32x4 wpost = a.w_post ? ld_row<DT, TAIL>(a.w_post, v, hidden) : ones(DT);
                    const u32x4 wpre = a.w_pre ? ld_row<DT, TAIL>(a.w_pre, v, hidden) : ones(DT);
                    const u32x4 gate = grow ? ld_row<DT, TAIL>(grow, v, hidden) : ones(DT);
                    const u32x4 res = row(a.residual, a.ld_residual), dhv = row(a.d_h, a.ld_d_h), dzv = row(a.d_z, a.ld_d_z);
                    float y[VE], h[VE], e[VE], pre[VE], unused[3] = {0.0f, 0.0f, 0.0f};
                    unpack<DT>(row(a.src[0], a.ld_src), y);
                    for (int r = 1; r < a.nsrc; ++r) {
                        float f[VE];
                        unpack<DT>(row(a.src[r], a.ld_src), f);
#pragma unroll
                        for (int k = 0; k < VE; ++k)
                            y[k] += f[k];
                    }
                    row_sums<DT, VE>(y, res, dhv, dzv, wpost, wpre, gate, p, q, a.residual_scale, h, e, pre,
                                     pass == 0 ? s : unused);
                    if (pass == 0)
                        continue;
                    float o1[VE], o2[VE], tt[VE];
                    row_results<DT, VE>(y, h, e, wpost, gate, p, m1, m2, a.residual_scale, o1, o2, tt);
                    // all of this vector's loads are over: d_residual may be d_h
                    if (a.d_residual)
                        st_row<DT, TAIL>(static_cast<char*>(a.d_residual) + t * a.ld_d_residual * EB, v, hidden, pack<DT>(o1));
                    st_row<DT, TAIL>(static_cast<char*>(a.d_src) + t * a.ld_d_src * EB, v, hidden, pack<DT>(o2));
                    float ot[VE] = {}, op[VE] = {};
                    if (t > s0)
                        ld_sums<VE>(to, v * VE, hidden, ot);
                    if (t > r0)
                        ld_sums<VE>(part_pre, v * VE, hidden, op);
#pragma unroll
                    for (int k = 0; k < VE; ++k) {
                        ot[k] += tt[k];
                        op[k] += pre[k];
                    }
                    st_sums<VE>(to, v * VE, hidden, ot);
                    st_sums<VE>(part_pre, v * VE, hidden, op);
                }
                if (pass == 0) {
                    block_sums<3, 1024 / kWave>(s, sums, turn);
                    row_means(a, s, p, q, m1, m2);
                }
            }
        }
        if constexpr (MULTI)
            for (int v = (int)threadIdx.x; v < nvec; v += 1024) {
                float w1[VE], g[VE];
                unpack<DT>(a.w_post ? ld_row<DT, TAIL>(a.w_post, v, hidden) : ones(DT), w1);
                unpack<DT>(grow ? ld_row<DT, TAIL>(grow, v, hidden) : ones(DT), g);
#pragma unroll
                for (int k = 0; k < VE; ++k) {
                    const int c = v * VE + k;
                    if (c < hidden) {
                        part_post[c] = s0 == r0 ? g[k] * to[c] : part_post[c] + g[k] * to[c];
                        to[c] = w1[k] * to[c];
                    }
                }
            }
        s0 = s1;
    }
}

// Adds the parts' sums in their order: 64 columns a workgroup, the parts
// dealt to 16 waves. blockIdx.y: T (or, with several gate rows, d_w_post),
// d_w_pre, then the gate's rows that cross parts.
template <int DT>
__global__ __launch_bounds__(1024) void k_norm_params(NormBwdArgs a)
{
    __shared__ float lds[16][64];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const size_t c = (size_t)blockIdx.x * 64 + lane;
    const float* from = blockIdx.y == 1 ? a.part_pre : a.part_post;
    size_t w0 = 0, w1 = a.parts, stride = a.hidden, g0 = 0;
    const size_t g = blockIdx.y < 2 ? 0 : blockIdx.y - 2;
    if (blockIdx.y >= 2) {
        g0 = g * a.gate_rows;
        const size_t g1 = g0 + a.gate_rows < a.rows ? g0 + a.gate_rows : a.rows;
        from = a.part_gate;
        stride = 2 * a.hidden;
        w0 = g0 / a.part_rows;
        w1 = (g1 - 1) / a.part_rows + 1;
        if (w1 - w0 == 1)
            return;   // written at once
    }
    float s = 0.0f;
    if (c < a.hidden)
#pragma unroll 8
        for (size_t w = w0 + wave; w < w1; w += 16) {
            const size_t slot = blockIdx.y >= 2 && g0 >= w * a.part_rows ? a.hidden : 0;
            s += from[w * stride + slot + c];
        }
    lds[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || c >= a.hidden)
        return;
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w)
        s += lds[w][lane];
    auto param = [&](const void* p) {
        if (!p)
            return 1.0f;
        if constexpr (DT == 0)
            return static_cast<const float*>(p)[c];
        else
            return bf16_lo(static_cast<const uint16_t*>(p)[c]);
    };
    if (blockIdx.y >= 2) {
        a.d_gate[g * a.hidden + c] = s;
    } else if (blockIdx.y == 1) {
        if (a.d_w_pre)
            a.d_w_pre[c] = s;
    } else {
        const bool one = a.gate_rows >= a.rows;   // s is T of all rows
        if (a.d_w_post)
            a.d_w_post[c] = one && a.rows ? param(a.gate) * s : s;
        if (one && a.rows && a.d_gate)
            a.d_gate[c] = param(a.w_post) * s;
    }
}

template <int DT, bool TAIL, int NV, int WG, int R, bool ACC>
const void* backward_of(bool multi)
{
    return multi ? (const void*)k_norm_backward<DT, TAIL, NV, WG, R, true, ACC>
                 : (const void*)k_norm_backward<DT, TAIL, NV, WG, R, false, ACC>;
}

template <int DT, bool TAIL>
const void* backward_fn(unsigned threads, unsigned teams, int nv, bool multi)
{
    if (threads == 64)
        return teams > 1 ? nv == 1 ? backward_of<DT, TAIL, 1, 512, 8, false>(multi) : backward_of<DT, TAIL, 2, 512, 8, false>(multi)
               : nv == 1 ? backward_of<DT, TAIL, 1, 64, 1, false>(multi)
                         : backward_of<DT, TAIL, 2, 64, 1, false>(multi);
    if (threads == 128)
        return backward_of<DT, TAIL, 2, 128, 1, false>(multi);
    if (threads == 256)
        return backward_of<DT, TAIL, 2, 256, 1, false>(multi);
    if (threads == 512)
        return nv <= 2 ? backward_of<DT, TAIL, 2, 512, 1, false>(multi) : backward_of<DT, TAIL, 3, 512, 1, DT == 1>(multi);
    if (nv <= 2)
        return backward_of<DT, TAIL, 2, 1024, 1, true>(multi);
    return multi ? (const void*)k_norm_backward_long<DT, TAIL, true> : (const void*)k_norm_backward_long<DT, TAIL, false>;
}

// How a call's rows are spread: `threads` and `nv` vectors a thread for a
// row, `teams` rows at a time in a workgroup, part_rows rows a workgroup.
struct Spread {
    unsigned threads, teams;
    int nv;
    size_t part_rows, parts;
};

// Rows of up to 128 vectors take a wave each, eight to a workgroup, so that
// there are few parts to add (unless a gate row has fewer than eight rows,
// which would leave teams idle); longer rows two vectors a thread. 512
// threads a CU: the loads ahead keep the memory busy, and every part costs
// its sums' write and read.
Spread spread(size_t rows, size_t hidden, size_t gate_rows, int dtype)
{
    Spread s;
    const size_t nvec = vectors(hidden, dtype);
    s.threads = nvec > 1024 && nvec <= 1536 ? 512 : threads_for((nvec + 1) / 2, 1024);
    s.nv = (int)((nvec + s.threads - 1) / s.threads);
    s.teams = s.threads == kWave && gate_rows >= 8 ? 8 : 1;
    const size_t wg = s.threads * s.teams;
    const size_t most = (size_t)device_cu_count() * (wg < 512 ? 512 / wg : 1);
    s.part_rows = (rows + most - 1) / most;
    if (s.part_rows < 1)
        s.part_rows = 1;
    // whole gate rows where they are shorter than a part: only longer ones cross
    if (gate_rows <= s.part_rows)
        s.part_rows = (s.part_rows + gate_rows - 1) / gate_rows * gate_rows;
    s.parts = (rows + s.part_rows - 1) / s.part_rows;
    return s;
}

}  // namespace

size_t norm_backward_parts(size_t rows, size_t hidden, size_t gate_rows)
{
    size_t most = 0;
    for (int dtype = 0; dtype < 2; ++dtype)
        for (size_t g : {gate_rows, rows < 1 ? 1 : rows}) {   // without a gate all rows share one
            const size_t p = spread(rows, hidden, g, dtype).parts;
            most = p > most ? p : most;
        }
    return most;
}

hipError_t launch_norm_backward(const NormBwdArgs& in, int dtype, hipStream_t s)
{
    NormBwdArgs a = in;
    void* params[] = {&a};
    if (!a.gate || a.gate_rows > a.rows)
        a.gate_rows = a.rows < 1 ? 1 : a.rows;
    const Spread sp = spread(a.rows, a.hidden, a.gate_rows, dtype);
    const bool tail = partial(a.hidden, dtype), multi = a.gate_rows < a.rows;
    a.part_rows = sp.part_rows;
    a.parts = sp.parts;
    a.part_pre = a.part_post + a.parts * a.hidden;
    a.part_gate = a.part_pre + a.parts * a.hidden;
    if (a.parts) {
        const void* fn = dtype == 0 ? tail ? backward_fn<0, true>(sp.threads, sp.teams, sp.nv, multi)
                                           : backward_fn<0, false>(sp.threads, sp.teams, sp.nv, multi)
                         : tail ? backward_fn<1, true>(sp.threads, sp.teams, sp.nv, multi)
                                : backward_fn<1, false>(sp.threads, sp.teams, sp.nv, multi);
        const hipError_t e = launch_logged("k_norm_backward", fn, dim3((unsigned)a.parts), dim3(sp.threads * sp.teams), params, s);
        if (e != hipSuccess)
            return e;
    }
    const bool cross = multi && a.d_gate && a.gate_rows > a.part_rows;
    const size_t groups = cross ? (a.rows + a.gate_rows - 1) / a.gate_rows : 0;
    if (!a.d_w_post && !a.d_w_pre && !a.d_gate)
        return hipSuccess;
    return launch_logged("k_norm_params", dtype ? (const void*)k_norm_params<1> : (const void*)k_norm_params<0>,
                         dim3((unsigned)((a.hidden + 63) / 64), (unsigned)(2 + groups)), dim3(1024), params, s);
}

}  // namespace rx
