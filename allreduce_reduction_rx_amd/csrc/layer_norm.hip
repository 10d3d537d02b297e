// layer_norm.hip -- the sum over the ranks with bias, dropout, residual and
// layer norm, and its gradient (gfx950). Defined in rx.h.
//
// Forward: one workgroup holds a row in registers, every input is read once and
// every output written once. The variance is that of the differences from the
// mean: a second sum over the row, but right for rows whose mean is large
// against their spread. HBM-bound.
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

template <class A>
__device__ __forceinline__ Dropper dropper(const A& a, size_t row)
{
    Dropper d = {};
    if (a.threshold) {
        d.seed = a.rng[0];
        d.offset = a.rng[1];
        d.first = row * ((a.hidden + 7) / 8);
        d.threshold = a.threshold;
    }
    return d;
}

// Loads ahead as in k_norm: with one vector a thread, everything before the
// sources.
template <int DT, bool TAIL, int NV, int WG>
__global__ __launch_bounds__(WG) void k_layer_norm(LayerNormArgs a)
{
    constexpr int VE = Elem<DT>::kVE, EB = Elem<DT>::kBytes;
    constexpr bool kAhead = NV == 1;
    __shared__ float lds[2 * 16];
    int turn = 0;
    const size_t t = blockIdx.x;
    const int hidden = (int)a.hidden, tid = (int)threadIdx.x, bd = (int)blockDim.x;
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
    fold_row<DT, TAIL, NV>(a.src, a.nsrc, t * a.ld_src * EB, hidden, y);
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
        const Dropper d = dropper(a, t);
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
    block_sums<1>(&s, lds, turn);
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
    block_sums<1>(&q, lds, turn);
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
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            s[0] += g[k];
            s[1] += g[k] * ((x[k] - mean) * rstd);
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
        if (a.threshold)
            drop_vector<DT>(dropper(a, t), v, a.gain, o);
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

// Adds the parts' sums in their order: 64 columns a workgroup, the parts
// dealt to 16 waves. blockIdx.y: d_w, d_b, d_bias.
__global__ __launch_bounds__(1024) void k_layer_norm_params(LayerNormBwdArgs a)
{
    __shared__ float lds[16][kWave];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const size_t c = (size_t)blockIdx.x * kWave + lane;
    float* to = blockIdx.y == 0 ? a.d_w : blockIdx.y == 1 ? a.d_b : a.d_bias;
    if (!to)
        return;
    float s = 0.0f;
    if (c < a.hidden)
#pragma unroll 8
        for (size_t w = wave; w < a.nparts; w += 16)
            s += a.parts[(w * 3 + blockIdx.y) * a.hidden + c];
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

template <int NV, int WG>
const void* forward_of(int dtype, bool tail)
{
    if (dtype == 0)
        return tail ? (const void*)k_layer_norm<0, true, NV, WG> : (const void*)k_layer_norm<0, false, NV, WG>;
    return tail ? (const void*)k_layer_norm<1, true, NV, WG> : (const void*)k_layer_norm<1, false, NV, WG>;
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

// Parts of the rows: about four workgroups a CU over all column blocks.
size_t column_parts(size_t rows, size_t hidden, int dtype)
{
    const size_t blocks = (vectors(hidden, dtype) + kWave - 1) / kWave, want = 4 * (size_t)device_cu_count();
    size_t parts = blocks ? (want + blocks - 1) / blocks : 1;
    const size_t most = (rows + 3) / 4;
    return parts < most ? parts : most;
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& in, int dtype, hipStream_t s)
{
    LayerNormArgs a = in;
    void* params[] = {&a};
    const size_t nvec = vectors(a.hidden, dtype);
    const unsigned wg = forward_threads(nvec, a.rows);
    return launch_logged("k_layer_norm", forward_fn(dtype, partial(a.hidden, dtype), wg, nvec), dim3((unsigned)a.rows), dim3(wg),
                         params, s);
}

// Floats: two a row, and three sums a column for each part (of either type).
size_t layer_norm_backward_floats(size_t rows, size_t hidden)
{
    const size_t p0 = column_parts(rows, hidden, 0), p1 = column_parts(rows, hidden, 1);
    return 2 * rows + 3 * hidden * (p0 > p1 ? p0 : p1);
}

hipError_t launch_layer_norm_backward(const LayerNormBwdArgs& in, int dtype, hipStream_t s)
{
    LayerNormBwdArgs a = in;
    void* params[] = {&a};
    const bool tail = partial(a.hidden, dtype);
    const size_t nvec = vectors(a.hidden, dtype);
    a.parts = a.means + 2 * a.rows;
    a.nparts = column_parts(a.rows, a.hidden, dtype);
    if (a.rows) {
        a.part_rows = (a.rows + a.nparts - 1) / a.nparts;
        a.nparts = (a.rows + a.part_rows - 1) / a.part_rows;
        if (a.d_z) {
            const void* fn = dtype == 0 ? tail ? (const void*)k_layer_norm_means<0, true> : (const void*)k_layer_norm_means<0, false>
                             : tail     ? (const void*)k_layer_norm_means<1, true>
                                        : (const void*)k_layer_norm_means<1, false>;
            const hipError_t e = launch_logged("k_layer_norm_means", fn, dim3((unsigned)a.rows), dim3(threads_for((nvec + 1) / 2, 1024)), params, s);
            if (e != hipSuccess)
                return e;
        }
        const void* fn = dtype == 0 ? tail ? (const void*)k_layer_norm_columns<0, true> : (const void*)k_layer_norm_columns<0, false>
                         : tail     ? (const void*)k_layer_norm_columns<1, true>
                                    : (const void*)k_layer_norm_columns<1, false>;
        const hipError_t e = launch_logged("k_layer_norm_columns", fn, dim3((unsigned)((nvec + kWave - 1) / kWave), (unsigned)a.nparts), dim3(256), params, s);
        if (e != hipSuccess)
            return e;
    }
    if (!a.d_w && !a.d_b && !a.d_bias)
        return hipSuccess;
    return launch_logged("k_layer_norm_params", (const void*)k_layer_norm_params, dim3((unsigned)((a.hidden + 63) / 64), 3), dim3(1024),
                         params, s);
}

}  // namespace rx
