// layer_norm.hip -- the sum over the ranks with bias, dropout, residual and
// layer norm, and its gradient (gfx950). Defined in rx.h.
//
// Forward: one workgroup holds a row in registers, every input is read once and
// every output written once. The variance is that of the differences from the
// mean: a second sum over the row, but right for rows whose mean is large
// against their spread. HBM-bound: 16384 x 8192 BF16 with two sources, residual,
// bias and dropout takes 220 us for 1.34 GB read and written (6.1 TB/s); the
// generator's 40 multiplications a vector run while the memory does.
#include "norm_common.hpp"
#include "philox.hpp"

namespace rx {
namespace {

// The elements of vector v that lie in the row, as a number.
template <int DT, bool TAIL>
__device__ __forceinline__ int inside(int v, int hidden)
{
    constexpr int VE = Elem<DT>::kVE;
    const int left = hidden - v * VE;
    return TAIL ? left : left > 0 ? VE : 0;
}

// The call's dropper: asked for at a kernel's start, long before it is used.
template <class A>
__device__ __forceinline__ Dropper dropper(const A& a)
{
    Dropper d = {};
    if (a.threshold) {
        d.seed = a.rng[0];
        d.offset = a.rng[1];
        d.threshold = a.threshold;
    }
    return d;
}
__device__ __forceinline__ void at_row(Dropper& d, size_t row, size_t hidden) { d.first = row * ((hidden + 7) / 8); }

// Loads ahead as in k_norm: with one vector a thread, everything before the
// sources. NARROW: a row has a.lanes of a wave's lanes, a power of two, and a wave
// 64 / a.lanes rows (16000 x 64 BF16 with residual, bias and dropout: 5.3 us, 11.9 with a
// workgroup a row).
template <int DT, bool TAIL, int NV, int WG, bool NARROW>
__global__ __launch_bounds__(WG) void k_layer_norm(LayerNormArgs a)
{
    constexpr int VE = Elem<DT>::kVE, EB = Elem<DT>::kBytes;
    constexpr bool kAhead = NV == 1;
    __shared__ float lds[2 * 16];
    int turn = 0;
    const int hidden = (int)a.hidden, bd = NARROW ? a.lanes : (int)blockDim.x;
    const int tid = NARROW ? (int)threadIdx.x & (bd - 1) : (int)threadIdx.x;
    size_t t = blockIdx.x;
    if (NARROW) {
        t = t * (WG / bd) + threadIdx.x / bd;
        if (t >= a.rows)   // whole groups of lanes, which share nothing with the others
            return;
    }
    auto row_sum = [&](float& v) {
        if (NARROW)
            v = group_sum_rt(v, bd);
        else
            block_sums<1>(&v, lds, turn);
    };
    Dropper d = dropper(a);
    u32x4 res[NV], wv[NV], bv[NV], biasv[NV];
    auto load = [&](u32x4* to, const void* row) {
#pragma unroll
        for (int u = 0; u < NV; ++u)
            to[u] = ld_raw<DT, TAIL>(row, tid + u * bd, hidden);
    };
    auto at = [&](const u32x4* from, int u, float* f) { unpack<DT>(fixed<DT, TAIL>(from[u], tid + u * bd, hidden), f); };
    if (a.residual)
#pragma unroll
        for (int u = 0; u < NV; ++u)
            res[u] = ld_raw<DT, TAIL, true>(static_cast<const char*>(a.residual) + t * a.ld_residual * EB, tid + u * bd, hidden);
    if (kAhead) {
        if (a.bias) load(biasv, a.bias);
        if (a.w) load(wv, a.w);
        if (a.b) load(bv, a.b);
    }
    float y[NV][VE];
    fold_row<DT, TAIL, NV>(a.src, a.nsrc, t * a.ld_src * EB, hidden, tid, bd, y);
    if (a.bias) {
        if (!kAhead) load(biasv, a.bias);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float f[VE];
            at(biasv, u, f);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                y[u][k] += f[k];
        }
    }
    if (a.threshold) {
        at_row(d, t, a.hidden);
#pragma unroll
        for (int u = 0; u < NV; ++u)
            drop_vector<DT>(d, tid + u * bd, a.gain, y[u]);
    }
    if (a.residual) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float f[VE];
            at(res, u, f);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                y[u][k] = f[k] + y[u][k];
        }
    }
    // h as it is stored
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const u32x4 h = pack<DT>(y[u]);
        unpack<DT>(h, y[u]);
        if (a.out_h)
            st_row<DT, TAIL, true>(static_cast<char*>(a.out_h) + t * a.ld_h * EB, tid + u * bd, hidden, h);
    }
    if (!a.out_z)
        return;
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int n = inside<DT, TAIL>(tid + u * bd, hidden);
#pragma unroll
        for (int k = 0; k < VE; ++k)
            s += k < n ? y[u][k] : 0.0f;
    }
    row_sum(s);
    const float mean = s * a.inv_hidden;
    float q = 0.0f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int n = inside<DT, TAIL>(tid + u * bd, hidden);
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            y[u][k] -= mean;
            q += k < n ? y[u][k] * y[u][k] : 0.0f;
        }
    }
    row_sum(q);
    const float rstd = 1.0f / __builtin_sqrtf(q * a.inv_hidden + a.eps);
    if (tid == 0) {
        if (a.mean)
            a.mean[t] = mean;
        if (a.rstd)
            a.rstd[t] = rstd;
    }
    if (!kAhead) {
        if (a.w) load(wv, a.w);
        if (a.b) load(bv, a.b);
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float f[VE];
#pragma unroll
        for (int k = 0; k < VE; ++k)
            y[u][k] *= rstd;
        if (a.w) {
            at(wv, u, f);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                y[u][k] *= f[k];
        }
        if (a.b) {
            at(bv, u, f);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                y[u][k] += f[k];
        }
        st_row<DT, TAIL, true>(static_cast<char*>(a.out_z) + t * a.ld_z * EB, tid + u * bd, hidden, pack<DT>(y[u]));
    }
}

// ---- gradient ------------------------------------------------------------------

// The two means of a row, mean(a) and mean(a x), into the workspace.
template <int DT, bool TAIL>
__global__ __launch_bounds__(1024) void k_layer_norm_means(LayerNormBwdArgs a)
{
    constexpr int VE = Elem<DT>::kVE, EB = Elem<DT>::kBytes;
    __shared__ float lds[2 * 16 * 2];
    int turn = 0;
    const size_t t = blockIdx.x;
    const int hidden = (int)a.hidden, nvec = (hidden + VE - 1) / VE;
    const void* h = static_cast<const char*>(a.h) + t * a.ld_h * EB;
    const void* dz = static_cast<const char*>(a.d_z) + t * a.ld_d_z * EB;
    const float mean = a.mean[t], rstd = a.rstd[t];
    float s[2] = {0.0f, 0.0f};
#pragma unroll 2
    for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
        float x[VE], g[VE], w[VE];
        unpack<DT>(ld_row<DT, TAIL>(h, v, hidden), x);
        unpack<DT>(ld_row<DT, TAIL>(dz, v, hidden), g);
        if (a.w) {
            unpack<DT>(ld_row<DT, TAIL>(a.w, v, hidden), w);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                g[k] *= w[k];
        }
        const int n = inside<DT, TAIL>(v, hidden);
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            s[0] += g[k];
            s[1] += g[k] * (k < n ? (x[k] - mean) * rstd : 0.0f);
        }
    }
    block_sums<2>(s, lds, turn);
    if (threadIdx.x == 0) {
        a.means[2 * t] = s[0] * a.inv_hidden;
        a.means[2 * t + 1] = s[1] * a.inv_hidden;
    }
}

// 64 vectors of the columns and a part of the rows a workgroup, its four waves
// a row each in turn; the parameters' sums of the part.
template <int DT, bool TAIL>
__global__ __launch_bounds__(256) void k_layer_norm_columns(LayerNormBwdArgs a)
{
    constexpr int VE = Elem<DT>::kVE, EB = Elem<DT>::kBytes;
    __shared__ float lds[4][VE][kWave];
    const int hidden = (int)a.hidden, lane = lane_id(), wave = threadIdx.x / kWave;
    const int v = (int)blockIdx.x * kWave + lane;
    const size_t r0 = blockIdx.y * a.part_rows, r1 = r0 + a.part_rows < a.rows ? r0 + a.part_rows : a.rows;
    Dropper d = dropper(a);
    float w[VE], acc[3][VE] = {};
#pragma unroll
    for (int k = 0; k < VE; ++k)
        w[k] = 1.0f;
    if (a.w)
        unpack<DT>(ld_row<DT, TAIL>(a.w, v, hidden), w);
    for (size_t t = r0 + wave; t < r1; t += 4) {
        float o[VE], dz[VE], x[VE];
#pragma unroll
        for (int k = 0; k < VE; ++k)
            o[k] = 0.0f;
        if (a.d_h)
            unpack<DT>(ld_row<DT, TAIL>(static_cast<const char*>(a.d_h) + t * a.ld_d_h * EB, v, hidden), o);
        if (a.d_z) {
            const float mean = a.mean[t], rstd = a.rstd[t], m1 = a.means[2 * t], m2 = a.means[2 * t + 1];
            unpack<DT>(ld_row<DT, TAIL>(static_cast<const char*>(a.h) + t * a.ld_h * EB, v, hidden), x);
            unpack<DT>(ld_row<DT, TAIL>(static_cast<const char*>(a.d_z) + t * a.ld_d_z * EB, v, hidden), dz);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                x[k] = (x[k] - mean) * rstd;
                acc[0][k] += dz[k] * x[k];
                acc[1][k] += dz[k];
                o[k] += rstd * (dz[k] * w[k] - m1 - x[k] * m2);
            }
        }
        if (a.d_residual)
            st_row<DT, TAIL, true>(static_cast<char*>(a.d_residual) + t * a.ld_d_residual * EB, v, hidden, pack<DT>(o));
        if (a.threshold) {
            at_row(d, t, a.hidden);
            drop_vector<DT>(d, v, a.gain, o);
        }
#pragma unroll
        for (int k = 0; k < VE; ++k)
            acc[2][k] += o[k];
        if (a.d_src)
            st_row<DT, TAIL, true>(static_cast<char*>(a.d_src) + t * a.ld_d_src * EB, v, hidden, pack<DT>(o));
    }
    if (!a.d_w && !a.d_b && !a.d_bias)
        return;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < VE; ++k)
            lds[wave][k][lane] = acc[p][k];
        __syncthreads();
        if (wave == 0)
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                const float s = ((lds[0][k][lane] + lds[1][k][lane]) + lds[2][k][lane]) + lds[3][k][lane];
                if (v * VE + k < hidden)
                    a.parts[((size_t)blockIdx.y * 3 + p) * a.hidden + v * VE + k] = s;
            }
    }
}

// A row's vectors in registers, its two sums across the threads that hold it, and
// the parameters' sums of a range of rows (a part) in registers too: every input is
// read once. Several teams of a.lanes lanes (a power of two up to a wave) have a row
// each where TEAMS; the next row's loads go out as soon as this row's are
// unpacked, before its sums and stores, and the next two rows' where a workgroup has a CU
// for itself (16384 x 8192 BF16 with dropout, forward and gradient 474 us, 486 with one; 8192 x 4096,
// two workgroups a CU, 89 and 87). 16384 x 8192 BF16 with dropout and all outputs: 250 us for
// 1.34 GB (5.4 TB/s), 340 by k_layer_norm_means and k_layer_norm_columns, which read h and
// d_z twice.
template <int DT, bool TAIL, int NV, int WG, bool TEAMS, bool DROP>
__global__ __launch_bounds__(WG, 2) void k_layer_norm_backward(LayerNormBwdArgs a)
{
    constexpr int VE = Elem<DT>::kVE, EB = Elem<DT>::kBytes, E = NV * VE;
    __shared__ float sums[2 * 16 * 2];
    __shared__ float join[TEAMS ? WG * VE : 1];
    int turn = 0;
    const int hidden = (int)a.hidden;
    const int W = TEAMS ? a.lanes : WG, R = WG / W, tid = TEAMS ? (int)threadIdx.x & (W - 1) : (int)threadIdx.x;
    const int team = TEAMS ? W == kWave ? (int)__builtin_amdgcn_readfirstlane(threadIdx.x / kWave) : (int)threadIdx.x / W : 0;
    const size_t r0 = blockIdx.x * a.part_rows, r1 = r0 + a.part_rows < a.rows ? r0 + a.part_rows : a.rows;
    const u32x4 zero = {0, 0, 0, 0};
    const uint32_t one = DT ? 0x3F803F80u : 0x3F800000u;
    Dropper d = {};
    if (DROP)
        d = dropper(a);
    constexpr int D = NV == 2 && WG == 512 && !TEAMS ? 2 : 1;   // rows ahead
    struct Row {
        u32x4 h[NV], dh[NV], dz[NV];
        float mean, rstd;
    } ahead[D];
    u32x4 w[NV];
    float acc_w[E] = {}, acc_b[E] = {}, acc_bias[E] = {};
#pragma unroll
    for (int u = 0; u < NV; ++u)
        w[u] = a.w ? ld_row<DT, TAIL>(a.w, tid + u * W, hidden) : u32x4{one, one, one, one};
    auto load = [&](Row& to, size_t t) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int v = tid + u * W;
            to.h[u] = a.d_z ? ld_raw<DT, TAIL, true, false>(static_cast<const char*>(a.h) + t * a.ld_h * EB, v, hidden) : zero;
            to.dz[u] = a.d_z ? ld_raw<DT, TAIL, true, false>(static_cast<const char*>(a.d_z) + t * a.ld_d_z * EB, v, hidden) : zero;
            to.dh[u] = a.d_h ? ld_raw<DT, TAIL, true, false>(static_cast<const char*>(a.d_h) + t * a.ld_d_h * EB, v, hidden) : zero;
        }
        to.mean = a.d_z ? a.mean[t] : 0.0f;
        to.rstd = a.d_z ? a.rstd[t] : 0.0f;
    };
    auto step = [&](Row& now, size_t t) {
        const float mean = now.mean, rstd = now.rstd;
        float x[NV][VE], g[NV][VE], o[NV][VE], s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float wf[VE];
            auto whole = [&](u32x4 y) { return fixed<DT, TAIL>(y, tid + u * W, hidden); };
            unpack<DT>(whole(now.h[u]), x[u]);
            unpack<DT>(whole(now.dz[u]), g[u]);
            unpack<DT>(whole(now.dh[u]), o[u]);
            unpack<DT>(w[u], wf);
            const int n = inside<DT, TAIL>(tid + u * W, hidden);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                // past the row d_z is 0, but mean rstd may be infinite
                x[u][k] = k < n ? (x[u][k] - mean) * rstd : 0.0f;
                acc_w[u * VE + k] = __builtin_fmaf(g[u][k], x[u][k], acc_w[u * VE + k]);
                acc_b[u * VE + k] += g[u][k];
                g[u][k] *= wf[k];
                s[0] += g[u][k];
                s[1] = __builtin_fmaf(g[u][k], x[u][k], s[1]);
            }
        }
        if (t + D * R < r1)
            load(now, t + D * R);
        if constexpr (TEAMS) {
            s[0] = group_sum_rt(s[0], W);
            s[1] = group_sum_rt(s[1], W);
        } else {
            block_sums<2, WG / kWave>(s, sums, turn);
        }
        const float m1 = s[0] * a.inv_hidden, m2 = s[1] * a.inv_hidden;
        if (DROP)
            at_row(d, t, a.hidden);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int v = tid + u * W;
#pragma unroll
            for (int k = 0; k < VE; ++k)
                o[u][k] = __builtin_fmaf(rstd, g[u][k] - m1 - x[u][k] * m2, o[u][k]);
            if (a.d_residual)
                st_row<DT, TAIL, true>(static_cast<char*>(a.d_residual) + t * a.ld_d_residual * EB, v, hidden, pack<DT>(o[u]));
            if (DROP)
                drop_vector<DT>(d, v, a.gain, o[u]);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                acc_bias[u * VE + k] += o[u][k];
            if (a.d_src)
                st_row<DT, TAIL, true>(static_cast<char*>(a.d_src) + t * a.ld_d_src * EB, v, hidden, pack<DT>(o[u]));
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (r0 + team + d * R < r1)
            load(ahead[d], r0 + team + d * R);
    for (size_t t = r0 + team; t < r1; t += D * R)
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (t + d * R < r1)
                step(ahead[d], t + d * R);
    if (!a.d_w && !a.d_b && !a.d_bias)
        return;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        float* acc = p == 0 ? acc_w : p == 1 ? acc_b : acc_bias;
        float* to = p == 0 ? a.d_w : p == 1 ? a.d_b : a.d_bias;
        if (!to)
            continue;
        if (a.nparts > 1)
            to = a.parts + (blockIdx.x * 3 + p) * a.hidden;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if constexpr (TEAMS) {   // a wave's teams, then the waves in their order
                const int wave = threadIdx.x / kWave, lane = lane_id();
                __syncthreads();
#pragma unroll
                for (int k = 0; k < VE; ++k)
                    join[(wave * VE + k) * kWave + lane] = across_rt(acc[u * VE + k], W);
                __syncthreads();
                if (team == 0)
#pragma unroll
                    for (int k = 0; k < VE; ++k) {
                        float v = join[k * kWave + lane];
#pragma unroll
                        for (int r = 1; r < WG / kWave; ++r)
                            v += join[(r * VE + k) * kWave + lane];
                        acc[u * VE + k] = v;
                    }
            }
            const int c = (tid + u * W) * VE;
            if (team == 0) {
#pragma unroll
                for (int k = 0; k < VE; k += 4)
                    if (c + k + 4 <= hidden)
                        st16_any(to + c + k, pack<0>(acc + u * VE + k));
                    else
                        for (int i = k; i < k + 4; ++i)
                            if (c + i < hidden)
                                to[c + i] = acc[u * VE + i];
            }
        }
    }
}

// Adds the parts' sums in their order: 64 columns a workgroup, the parts dealt
// to 16 waves, eight of a wave's loads at a time. blockIdx.y: d_w, d_b, d_bias.
__global__ __launch_bounds__(1024) void k_layer_norm_params(LayerNormBwdArgs a)
{
    __shared__ float lds[16][kWave];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const size_t c = (size_t)blockIdx.x * kWave + lane;
    float* to = blockIdx.y == 0 ? a.d_w : blockIdx.y == 1 ? a.d_b : a.d_bias;
    if (!to)
        return;
    const float* at = a.parts + blockIdx.y * a.hidden + (c < a.hidden ? c : 0);
    float s = 0.0f;
    for (size_t w0 = wave; w0 < a.nparts; w0 += 128) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const size_t w = w0 + 16 * i;
            x[i] = at[(w < a.nparts ? w : w0) * 3 * a.hidden];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s += w0 + 16 * i < a.nparts ? x[i] : 0.0f;
    }
    lds[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || c >= a.hidden)
        return;
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w)
        s += lds[w][lane];
    to[c] = s;
}

template <int NV, int WG, bool NARROW = false>
const void* forward_of(int dtype, bool tail)
{
    if (dtype == 0)
        return tail ? (const void*)k_layer_norm<0, true, NV, WG, NARROW> : (const void*)k_layer_norm<0, false, NV, WG, NARROW>;
    if constexpr (NV > 4)
        return nullptr;   // 32768 elements are four vectors a thread
    else
        return tail ? (const void*)k_layer_norm<1, true, NV, WG, NARROW> : (const void*)k_layer_norm<1, false, NV, WG, NARROW>;
}
const void* forward_fn(int dtype, bool tail, unsigned wg, size_t nvec)
{
    const size_t nv = (nvec + wg - 1) / wg;
    if (wg <= 256)
        return nv <= 1 ? forward_of<1, 256>(dtype, tail) : forward_of<2, 256>(dtype, tail);
    return nv <= 1   ? forward_of<1, 1024>(dtype, tail)
           : nv <= 2 ? forward_of<2, 1024>(dtype, tail)
           : nv <= 4 ? forward_of<4, 1024>(dtype, tail)
                     : forward_of<8, 1024>(dtype, tail);
}

// As for k_norm: two vectors a thread, one where there are no more rows than
// CUs; whole waves.
unsigned forward_threads(size_t nvec, size_t rows)
{
    const size_t per = rows <= (size_t)device_cu_count() ? 1 : 2, t = (nvec + per - 1) / per;
    return t >= 1024 ? 1024u : t < kWave ? (unsigned)kWave : (unsigned)((t + kWave - 1) / kWave * kWave);
}

// Lanes of a row of up to a wave's vectors: the next power of two.
int narrow_lanes(size_t nvec)
{
    int g = 1;
    while (g < kWave && (size_t)g < nvec)
        g *= 2;
    return g;
}

// How a gradient's rows are spread. Rows of up to 128 vectors take a wave's lanes or
// fewer, in workgroups of 512 threads; longer ones two vectors a thread, and workgroups of 512 threads a
// CU or one larger one: every part costs its sums' write and read. Rows beyond
// what the registers hold (1024 vectors BF16, FP32 2048) go by columns in parts, and
// rows shorter than a vector, whose loads would take the others' speed (1111 x 5001
// FP32 with dropout: 36 us with their code in the loop, 28 without).
struct Spread {
    bool whole;                // k_layer_norm_backward
    unsigned threads, lanes;   // of a workgroup; of a row where it has several, else 0
    int nv;                    // vectors a thread
    size_t part_rows, parts;
};
Spread spread(size_t rows, size_t hidden, int dtype)
{
    Spread s = {};
    const size_t nvec = vectors(hidden, dtype), cus = (size_t)device_cu_count();
    s.whole = hidden >= (dtype ? 8 : 4) && nvec <= (dtype ? 1024 : 2048);
    size_t want;
    if (s.whole) {
        s.threads = threads_for((nvec + 1) / 2, 512);
        s.nv = (int)((nvec + s.threads - 1) / s.threads);
        size_t teams = 1;
        if (s.threads == kWave) {
            s.threads = 512;
            s.lanes = (unsigned)narrow_lanes(nvec);
            teams = 512 / s.lanes;
        }
        want = cus * ((s.lanes && s.nv == 1 ? 1024 : 512) / s.threads);   // what the registers leave room for
        // every team a row, and up to two rows each one part, whose sums need no second launch
        if (want > (rows + teams - 1) / teams)
            want = (rows + teams - 1) / teams;
        if (rows <= 2 * teams)
            want = 1;
    } else {
        const size_t blocks = nvec ? (nvec + kWave - 1) / kWave : 1;   // about four workgroups a CU over all columns
        want = (4 * cus + blocks - 1) / blocks;
        if (want > (rows + 3) / 4)
            want = (rows + 3) / 4;
    }
    if (want < 1)
        want = 1;
    s.part_rows = (rows + want - 1) / want;
    if (s.part_rows < 1)
        s.part_rows = 1;
    s.parts = (rows + s.part_rows - 1) / s.part_rows;
    return s;
}

template <int DT, bool TAIL, bool DROP>
const void* backward_fn(const Spread& s)
{
    if (s.lanes)
        return s.nv == 1 ? (const void*)k_layer_norm_backward<DT, TAIL, 1, 512, true, DROP> : (const void*)k_layer_norm_backward<DT, TAIL, 2, 512, true, DROP>;
    if (s.threads == 128)
        return (const void*)k_layer_norm_backward<DT, TAIL, 2, 128, false, DROP>;
    if (s.threads == 256)
        return (const void*)k_layer_norm_backward<DT, TAIL, 2, 256, false, DROP>;
    if constexpr (DT == 0)
        if (s.nv > 2)
            return s.nv == 3 ? (const void*)k_layer_norm_backward<DT, TAIL, 3, 512, false, DROP> : (const void*)k_layer_norm_backward<DT, TAIL, 4, 512, false, DROP>;
    return (const void*)k_layer_norm_backward<DT, TAIL, 2, 512, false, DROP>;
}
template <int DT>
const void* backward_fn(const Spread& s, bool tail, bool drop)
{
    return tail ? drop ? backward_fn<DT, true, true>(s) : backward_fn<DT, true, false>(s)
                : drop ? backward_fn<DT, false, true>(s) : backward_fn<DT, false, false>(s);
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& in, int dtype, hipStream_t s)
{
    LayerNormArgs a = in;
    void* params[] = {&a};
    const size_t nvec = vectors(a.hidden, dtype);
    if (nvec <= kWave) {   // several rows a workgroup
        a.lanes = narrow_lanes(nvec);
        const size_t per = 256 / (size_t)a.lanes;
        return launch_logged("k_layer_norm", forward_of<1, 256, true>(dtype, partial(a.hidden, dtype)),
                             dim3((unsigned)((a.rows + per - 1) / per)), dim3(256), params, s);
    }
    const unsigned wg = forward_threads(nvec, a.rows);
    return launch_logged("k_layer_norm", forward_fn(dtype, partial(a.hidden, dtype), wg, nvec), dim3((unsigned)a.rows), dim3(wg),
                         params, s);
}

// Floats: two a row, and three sums a column for each part (of either type).
size_t layer_norm_backward_floats(size_t rows, size_t hidden)
{
    const size_t p0 = spread(rows, hidden, 0).parts, p1 = spread(rows, hidden, 1).parts;
    return (2 * rows + 3) / 4 * 4 + 3 * hidden * (p0 > p1 ? p0 : p1);
}

hipError_t launch_layer_norm_backward(const LayerNormBwdArgs& in, int dtype, hipStream_t s)
{
    LayerNormBwdArgs a = in;
    void* params[] = {&a};
    const bool tail = partial(a.hidden, dtype);
    const size_t nvec = vectors(a.hidden, dtype);
    const Spread sp = spread(a.rows, a.hidden, dtype);
    a.parts = a.means + (2 * a.rows + 3) / 4 * 4;
    a.nparts = sp.parts;
    a.part_rows = sp.part_rows;
    a.lanes = (int)sp.lanes;
    hipError_t e = hipSuccess;
    if (a.rows && sp.whole) {
        const void* fn = dtype == 0 ? backward_fn<0>(sp, tail, a.threshold) : backward_fn<1>(sp, tail, a.threshold);
        e = launch_logged("k_layer_norm_backward", fn, dim3((unsigned)sp.parts), dim3(sp.threads), params, s);
    } else if (a.rows) {
        if (a.d_z) {
            const void* fn = dtype == 0 ? tail ? (const void*)k_layer_norm_means<0, true> : (const void*)k_layer_norm_means<0, false>
                             : tail     ? (const void*)k_layer_norm_means<1, true>
                                        : (const void*)k_layer_norm_means<1, false>;
            e = launch_logged("k_layer_norm_means", fn, dim3((unsigned)a.rows), dim3(threads_for((nvec + 1) / 2, 1024)), params, s);
            if (e != hipSuccess)
                return e;
        }
        const void* fn = dtype == 0 ? tail ? (const void*)k_layer_norm_columns<0, true> : (const void*)k_layer_norm_columns<0, false>
                         : tail     ? (const void*)k_layer_norm_columns<1, true>
                                    : (const void*)k_layer_norm_columns<1, false>;
        e = launch_logged("k_layer_norm_columns", fn, dim3((unsigned)((nvec + kWave - 1) / kWave), (unsigned)sp.parts), dim3(256), params, s);
    }
    if (e != hipSuccess || (!a.d_w && !a.d_b && !a.d_bias) || (sp.whole && sp.parts == 1))
        return e;
    return launch_logged("k_layer_norm_params", (const void*)k_layer_norm_params, dim3((unsigned)((a.hidden + 63) / 64), 3), dim3(1024),
                         params, s);
}

}  // namespace rx
