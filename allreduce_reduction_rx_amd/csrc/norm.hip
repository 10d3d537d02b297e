// norm.hip -- the sum over the ranks fused with the norms, the gate and the
// residual around a block, and its gradient (gfx950). Defined in rx.h.
//
// One workgroup holds a row in registers, so every input is read once and
// every output written once: the sums for the two norms are the only thing
// that crosses lanes. HBM-bound (a few flops a byte).
#include "block_common.hpp"

namespace rx {
namespace {

// Sums of c[0 .. N) over the workgroup, the same in every thread. `lds`
// holds 2 x 16 x N floats, used in halves by turns, so one barrier a call is
// enough: a half is written again only after the next call's barrier.
template <int N>
__device__ __forceinline__ void block_sums(float* c, float* lds, int& turn)
{
    const int nw = blockDim.x / kWave;
#pragma unroll
    for (int j = 0; j < N; ++j)
        c[j] = wave_sum(c[j]);
    if (nw == 1)
        return;
    float* p = lds + turn * 16 * N;
    turn ^= 1;
    if (lane_id() == 0)
#pragma unroll
        for (int j = 0; j < N; ++j)
            p[(threadIdx.x / kWave) * N + j] = c[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j)
        c[j] = 0.0f;
    for (int w = 0; w < nw; ++w)
#pragma unroll
        for (int j = 0; j < N; ++j)
            c[j] += p[w * N + j];
}

// y (+)= sources r .. r + B - 1, in order; all B loads of a vector first.
template <int DT, bool TAIL, int NV, int B, bool FIRST>
__device__ __forceinline__ void fold_batch(const void* const* src, int r, size_t row_bytes, int hidden,
                                           float (*y)[Elem<DT>::kVE])
{
    constexpr int VE = Elem<DT>::kVE;
    u32x4 x[B][NV];
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
        for (int u = 0; u < NV; ++u)
            x[b][u] = ld_row<DT, TAIL, true>(static_cast<const char*>(src[r + b]) + row_bytes,
                                             (int)threadIdx.x + u * (int)blockDim.x, hidden);
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float f[VE];
            unpack<DT>(x[b][u], f);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                y[u][k] = FIRST && b == 0 ? f[k] : y[u][k] + f[k];
        }
}

template <int DT, bool TAIL, int NV>
__device__ __forceinline__ void fold_row(const void* const* src, int nsrc, size_t row_bytes, int hidden,
                                         float (*y)[Elem<DT>::kVE])
{
    int r;
    switch (nsrc) {
    case 1: fold_batch<DT, TAIL, NV, 1, true>(src, 0, row_bytes, hidden, y); return;
    case 2: fold_batch<DT, TAIL, NV, 2, true>(src, 0, row_bytes, hidden, y); return;
    case 3: fold_batch<DT, TAIL, NV, 3, true>(src, 0, row_bytes, hidden, y); return;
    default: fold_batch<DT, TAIL, NV, 4, true>(src, 0, row_bytes, hidden, y); r = 4;
    }
    for (; r + 4 <= nsrc; r += 4)
        fold_batch<DT, TAIL, NV, 4, false>(src, r, row_bytes, hidden, y);
    for (; r < nsrc; ++r)
        fold_batch<DT, TAIL, NV, 1, false>(src, r, row_bytes, hidden, y);
}

template <int DT, bool TAIL, int NV, int WG>
__global__ __launch_bounds__(WG) void k_norm(NormArgs a)
{
    constexpr int VE = Elem<DT>::kVE, EB = Elem<DT>::kBytes;
    __shared__ float lds[2 * 16];
    int turn = 0;
    const size_t t = blockIdx.x;
    const int hidden = (int)a.hidden;
    float y[NV][VE];
    fold_row<DT, TAIL, NV>(a.src, a.nsrc, t * a.ld_src * EB, hidden, y);
    u32x4 res[NV];
    if (a.residual)
#pragma unroll
        for (int u = 0; u < NV; ++u)
            res[u] = ld_row<DT, TAIL, true>(static_cast<const char*>(a.residual) + t * a.ld_residual * EB,
                                            (int)threadIdx.x + u * (int)blockDim.x, hidden);
    if (a.w_post) {
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
            for (int k = 0; k < VE; ++k)
                s += y[u][k] * y[u][k];
        block_sums<1>(&s, lds, turn);
        const float p = 1.0f / __builtin_sqrtf(s * a.inv_hidden + a.eps);
        if (a.rstd_post && threadIdx.x == 0)
            a.rstd_post[t] = p;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float w[VE];
            unpack<DT>(ld_row<DT, TAIL>(a.w_post, (int)threadIdx.x + u * (int)blockDim.x, hidden), w);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                y[u][k] = y[u][k] * p * w[k];
        }
    }
    if (a.gate) {
        const char* grow = static_cast<const char*>(a.gate) + t / a.gate_rows * a.hidden * EB;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float g[VE];
            unpack<DT>(ld_row<DT, TAIL>(grow, (int)threadIdx.x + u * (int)blockDim.x, hidden), g);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                y[u][k] *= g[k];
        }
    }
    if (a.residual) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float f[VE];
            unpack<DT>(res[u], f);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                y[u][k] += a.residual_scale * f[k];
        }
    }
    if (a.out_h) {
#pragma unroll
        for (int u = 0; u < NV; ++u)
            st_row<DT, TAIL, true>(static_cast<char*>(a.out_h) + t * a.ld_h * EB,
                                   (int)threadIdx.x + u * (int)blockDim.x, hidden, pack<DT>(y[u]));
    }
    if (!a.out_z)
        return;
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int k = 0; k < VE; ++k)
            s += y[u][k] * y[u][k];
    block_sums<1>(&s, lds, turn);
    const float q = 1.0f / __builtin_sqrtf(s * a.inv_hidden + a.eps);
    if (a.rstd_pre && threadIdx.x == 0)
        a.rstd_pre[t] = q;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float w[VE];
        unpack<DT>(ld_row<DT, TAIL>(a.w_pre, (int)threadIdx.x + u * (int)blockDim.x, hidden), w);
#pragma unroll
        for (int k = 0; k < VE; ++k)
            w[k] = y[u][k] * q * w[k];
        st_row<DT, TAIL, true>(static_cast<char*>(a.out_z) + t * a.ld_z * EB,
                               (int)threadIdx.x + u * (int)blockDim.x, hidden, pack<DT>(w));
    }
}

// Row range of a workgroup, its parameters' sums in registers. A gate row
// whose rows all lie in the range is written at once; one that crosses the
// range's start goes to slot 0 of the workgroup's two, one that only crosses
// its end to slot 1, and k_norm_params adds the slots in the rows' order.
//
// With e = d_h + q a, c = g w_post and dH = e - h q^3 S1 / H, where
// S1 = sum a h, the second mean is sum(c dH y) / H =
// (S2 - q^3 (S1 / H) S3) / H with S2 = sum c e y, S3 = sum c h y: the three
// sums cross the workgroup together.
template <int DT, bool TAIL, int NV, int WG>
__global__ __launch_bounds__(WG) void k_norm_backward(NormBwdArgs a)
{
    constexpr int VE = Elem<DT>::kVE, EB = Elem<DT>::kBytes;
    __shared__ float lds[2 * 16 * 3];
    int turn = 0;
    const int hidden = (int)a.hidden, bd = (int)blockDim.x, tid = (int)threadIdx.x;
    const size_t r0 = blockIdx.x * a.part_rows;
    const size_t r1 = r0 + a.part_rows < a.rows ? r0 + a.part_rows : a.rows;

    float acc_post[NV][VE] = {}, acc_pre[NV][VE] = {}, acc_gate[NV][VE] = {};
    u32x4 wpost[NV], wpre[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        if (a.w_post)
            wpost[u] = ld_row<DT, TAIL>(a.w_post, tid + u * bd, hidden);
        if (a.w_pre)
            wpre[u] = ld_row<DT, TAIL>(a.w_pre, tid + u * bd, hidden);
    }
    for (size_t t = r0; t < r1; ++t) {
        float y[NV][VE];
        fold_row<DT, TAIL, NV>(a.src, a.nsrc, t * a.ld_src * EB, hidden, y);
        u32x4 rv[NV], dhv[NV], dzv[NV], gv[NV];
        const size_t grp = a.gate ? t / a.gate_rows : 0;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int v = tid + u * bd;
            if (a.residual)
                rv[u] = ld_row<DT, TAIL, true>(static_cast<const char*>(a.residual) + t * a.ld_residual * EB, v, hidden);
            if (a.d_h)
                dhv[u] = ld_row<DT, TAIL, true>(static_cast<const char*>(a.d_h) + t * a.ld_d_h * EB, v, hidden);
            if (a.d_z)
                dzv[u] = ld_row<DT, TAIL, true>(static_cast<const char*>(a.d_z) + t * a.ld_d_z * EB, v, hidden);
            if (a.gate)
                gv[u] = ld_row<DT, TAIL>(static_cast<const char*>(a.gate) + grp * a.hidden * EB, v, hidden);
        }
        const float p = a.w_post ? a.rstd_post[t] : 1.0f;
        const float q = a.d_z ? a.rstd_pre[t] : 0.0f;

        float h[NV][VE], e[NV][VE], s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float w1[VE], w2[VE], g[VE], f[VE], dz[VE], dh[VE];
            if (a.w_post) unpack<DT>(wpost[u], w1);
            if (a.w_pre) unpack<DT>(wpre[u], w2);
            if (a.gate) unpack<DT>(gv[u], g);
            if (a.residual) unpack<DT>(rv[u], f);
            if (a.d_z) unpack<DT>(dzv[u], dz);
            if (a.d_h) unpack<DT>(dhv[u], dh);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                float c = a.gate ? g[k] : 1.0f;
                float uu = a.w_post ? y[u][k] * p * w1[k] : y[u][k];
                h[u][k] = c * uu + (a.residual ? a.residual_scale * f[k] : 0.0f);
                if (a.w_post) c *= w1[k];
                const float av = a.d_z ? dz[k] * w2[k] : 0.0f;
                if (a.d_z) acc_pre[u][k] += dz[k] * (h[u][k] * q);
                e[u][k] = (a.d_h ? dh[k] : 0.0f) + q * av;
                s[0] += av * h[u][k];
                s[1] += c * e[u][k] * y[u][k];
                s[2] += c * h[u][k] * y[u][k];
            }
        }
        block_sums<3>(s, lds, turn);
        const float m1 = q * q * q * (s[0] * a.inv_hidden);
        const float m2 = a.w_post ? p * p * ((s[1] - m1 * s[2]) * a.inv_hidden) : 0.0f;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float w1[VE], g[VE], o1[VE], o2[VE];
            if (a.w_post) unpack<DT>(wpost[u], w1);
            if (a.gate) unpack<DT>(gv[u], g);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                const float dH = e[u][k] - h[u][k] * m1;
                o1[k] = a.residual_scale * dH;
                const float uu = a.w_post ? y[u][k] * p * w1[k] : y[u][k];
                if (a.gate) acc_gate[u][k] += dH * uu;
                const float du = a.gate ? dH * g[k] : dH;
                if (a.w_post) {
                    acc_post[u][k] += du * (y[u][k] * p);
                    o2[k] = p * (du * w1[k] - y[u][k] * m2);
                } else {
                    o2[k] = du;
                }
            }
            const int v = tid + u * bd;
            if (a.d_residual)
                st_row<DT, TAIL, true>(static_cast<char*>(a.d_residual) + t * a.ld_d_residual * EB, v, hidden, pack<DT>(o1));
            st_row<DT, TAIL, true>(static_cast<char*>(a.d_src) + t * a.ld_d_src * EB, v, hidden, pack<DT>(o2));
        }
        if (a.d_gate && (t + 1 == r1 || (t + 1) % a.gate_rows == 0)) {
            const size_t g0 = grp * a.gate_rows;
            const size_t g1 = g0 + a.gate_rows < a.rows ? g0 + a.gate_rows : a.rows;
            float* to = g0 >= r0 && g1 <= r1 ? a.d_gate + grp * a.hidden
                                             : a.part_gate + (blockIdx.x * 2 + (g0 < r0 ? 0 : 1)) * a.hidden;
#pragma unroll
            for (int u = 0; u < NV; ++u)
#pragma unroll
                for (int k = 0; k < VE; ++k) {
                    const int c = (tid + u * bd) * VE + k;
                    if (c < hidden)
                        to[c] = acc_gate[u][k];
                    acc_gate[u][k] = 0.0f;
                }
        }
    }
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            const int c = (tid + u * bd) * VE + k;
            if (c < hidden) {
                if (a.d_w_post)
                    a.part_post[blockIdx.x * a.hidden + c] = acc_post[u][k];
                if (a.d_w_pre)
                    a.part_pre[blockIdx.x * a.hidden + c] = acc_pre[u][k];
            }
        }
}

// Adds the workgroups' partial sums in their order: 64 columns a workgroup,
// the parts dealt to 16 waves. blockIdx.y: d_w_post, d_w_pre, then the gate's
// rows that cross workgroups.
__global__ __launch_bounds__(1024) void k_norm_params(NormBwdArgs a)
{
    __shared__ float lds[16][64];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const size_t c = (size_t)blockIdx.x * 64 + lane;
    const float* from;
    float* to;
    size_t w0 = 0, w1 = a.parts, stride = a.hidden, g0 = 0;
    if (blockIdx.y == 0) {
        from = a.part_post;
        to = a.d_w_post;
    } else if (blockIdx.y == 1) {
        from = a.part_pre;
        to = a.d_w_pre;
    } else {
        const size_t g = blockIdx.y - 2;
        g0 = g * a.gate_rows;
        const size_t g1 = g0 + a.gate_rows < a.rows ? g0 + a.gate_rows : a.rows;
        from = a.part_gate;
        to = a.d_gate ? a.d_gate + g * a.hidden : nullptr;
        stride = 2 * a.hidden;
        w0 = g0 / a.part_rows;
        w1 = (g1 - 1) / a.part_rows + 1;
        if (w1 - w0 == 1)
            return;   // written at once
    }
    if (!to)
        return;
    float s = 0.0f;
    if (c < a.hidden)
        for (size_t w = w0 + wave; w < w1; w += 16) {
            const size_t slot = blockIdx.y >= 2 && g0 >= w * a.part_rows ? a.hidden : 0;
            s += from[w * stride + slot + c];
        }
    lds[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < a.hidden) {
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < 16; ++w)
            s += lds[w][lane];
        to[c] = s;
    }
}


#define RX_NORM_PICK(NAME)                                                                           \
    template <int NV, int WG>                                                                        \
    const void* NAME##_of(int dtype, bool tail)                                                      \
    {                                                                                                \
        if (dtype == 0)                                                                              \
            return tail ? (const void*)NAME<0, true, NV, WG> : (const void*)NAME<0, false, NV, WG>;  \
        return tail ? (const void*)NAME<1, true, NV, WG> : (const void*)NAME<1, false, NV, WG>;      \
    }                                                                                                \
    const void* NAME##_fn(int dtype, bool tail, unsigned wg, size_t nvec)                            \
    {                                                                                                \
        const size_t nv = (nvec + wg - 1) / wg;                                                      \
        if (wg <= 256)                                                                               \
            return nv <= 1 ? NAME##_of<1, 256>(dtype, tail) : NAME##_of<2, 256>(dtype, tail);        \
        return nv <= 1   ? NAME##_of<1, 1024>(dtype, tail)                                           \
               : nv <= 2 ? NAME##_of<2, 1024>(dtype, tail)                                           \
               : nv <= 4 ? NAME##_of<4, 1024>(dtype, tail)                                           \
                         : NAME##_of<8, 1024>(dtype, tail);                                          \
    }
RX_NORM_PICK(k_norm)
RX_NORM_PICK(k_norm_backward)
#undef RX_NORM_PICK

// Two vectors a thread where up to 1024 threads allow it.
unsigned norm_threads(size_t nvec) { return threads_for((nvec + 1) / 2, 1024); }

}  // namespace

hipError_t launch_norm(const NormArgs& in, int dtype, hipStream_t s)
{
    NormArgs a = in;
    void* params[] = {&a};
    const size_t nvec = vectors(a.hidden, dtype);
    const unsigned wg = norm_threads(nvec);
    return launch_logged("k_norm", k_norm_fn(dtype, partial(a.hidden, dtype), wg, nvec), dim3((unsigned)a.rows), dim3(wg),
                         params, s);
}

// About one workgroup a CU; whole gate rows where they are shorter than a
// workgroup's range, so that only longer ones cross workgroups.
void norm_backward_parts(size_t rows, size_t gate_rows, size_t* part_rows, size_t* parts)
{
    const size_t cus = (size_t)device_cu_count();
    size_t pr = (rows + cus - 1) / cus;
    if (pr < 1)
        pr = 1;
    if (gate_rows <= pr)
        pr = (pr + gate_rows - 1) / gate_rows * gate_rows;
    *part_rows = pr;
    *parts = (rows + pr - 1) / pr;
}

hipError_t launch_norm_backward(const NormBwdArgs& in, int dtype, hipStream_t s)
{
    NormBwdArgs a = in;
    void* params[] = {&a};
    const size_t nvec = vectors(a.hidden, dtype);
    const unsigned wg = norm_threads(nvec);
    if (a.parts) {
        const hipError_t e = launch_logged("k_norm_backward", k_norm_backward_fn(dtype, partial(a.hidden, dtype), wg, nvec),
                                           dim3((unsigned)a.parts), dim3(wg), params, s);
        if (e != hipSuccess)
            return e;
    }
    const bool cross = a.d_gate && a.gate_rows > a.part_rows;
    const size_t groups = cross ? (a.rows + a.gate_rows - 1) / a.gate_rows : 0;
    if (!a.d_w_post && !a.d_w_pre && !cross)
        return hipSuccess;
    return launch_logged("k_norm_params", (const void*)k_norm_params, dim3((unsigned)((a.hidden + 63) / 64), (unsigned)(2 + groups)),
                         dim3(1024), params, s);
}

}  // namespace rx
