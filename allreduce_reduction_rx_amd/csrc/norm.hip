// norm.hip -- the sum over the ranks fused with the norms, the gate and the
// residual around a block (gfx950). Defined in rx.h.
//
// One workgroup holds a row in registers, so every input is read once and
// every output written once: the sums for the two norms are the only thing
// that crosses lanes. HBM-bound (a few flops a byte).
#include "norm_common.hpp"

namespace rx {
namespace {

// y = the sources' sum in their order, B sources' loads of a thread in flight
// together.
template <int DT, bool TAIL, int NV>
__device__ __forceinline__ void fold_row(const void* const* src, int nsrc, size_t row_bytes, int hidden,
                                         float (*y)[Elem<DT>::kVE])
{
    constexpr int VE = Elem<DT>::kVE, B = NV == 1 ? 8 : 4;   // more would cost a longer row its occupancy
    const int tid = (int)threadIdx.x, bd = (int)blockDim.x;
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int k = 0; k < VE; ++k)
            y[u][k] = -0.0f;   // x + -0 = x for every x
    auto batch = [&](int r) {
        u32x4 x[B][NV];
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (r + b < nsrc)
#pragma unroll
                for (int u = 0; u < NV; ++u)
                    x[b][u] = ld_raw<DT, TAIL, true>(static_cast<const char*>(src[r + b]) + row_bytes, tid + u * bd, hidden);
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (r + b < nsrc)
#pragma unroll
                for (int u = 0; u < NV; ++u) {
                    float f[VE];
                    unpack<DT>(fixed<DT, TAIL>(x[b][u], tid + u * bd, hidden), f);
#pragma unroll
                    for (int k = 0; k < VE; ++k)
                        y[u][k] += f[k];
                }
    };
    batch(0);   // its pointers come with the kernel's arguments
#pragma unroll 1
    for (int r = B; r < nsrc; r += B)
        batch(r);
}

// NV 1: the gate and the weights are loaded before the sources too, so that a
// row has one round trip to memory (32 rows of 8192 BF16 over 8 sources: 6.0
// us, 6.6 with two vectors a thread and the weights loaded where they are
// used). With more rows than CUs the registers are worth more as occupancy
// (16384 x 8192 over two sources: 222 against 234 us).
template <int DT, bool TAIL, int NV, int WG>
__global__ __launch_bounds__(WG) void k_norm(NormArgs a)
{
    constexpr int VE = Elem<DT>::kVE, EB = Elem<DT>::kBytes;
    constexpr bool kAhead = NV == 1;
    __shared__ float lds[2 * 16];
    int turn = 0;
    const size_t t = blockIdx.x;
    const int hidden = (int)a.hidden, tid = (int)threadIdx.x, bd = (int)blockDim.x;
    const char* grow = a.gate ? static_cast<const char*>(a.gate) + t / a.gate_rows * a.hidden * EB : nullptr;
    u32x4 res[NV], wpost[NV], wpre[NV], gv[NV];
    auto load = [&](u32x4* to, const void* row) {
#pragma unroll
        for (int u = 0; u < NV; ++u)
            to[u] = ld_raw<DT, TAIL>(row, tid + u * bd, hidden);
    };
    if (a.residual)
#pragma unroll
        for (int u = 0; u < NV; ++u)
            res[u] = ld_raw<DT, TAIL, true>(static_cast<const char*>(a.residual) + t * a.ld_residual * EB, tid + u * bd, hidden);
    if (kAhead) {
        if (a.w_post) load(wpost, a.w_post);
        if (grow) load(gv, grow);
        if (a.out_z) load(wpre, a.w_pre);
    }
    float y[NV][VE];
    fold_row<DT, TAIL, NV>(a.src, a.nsrc, t * a.ld_src * EB, hidden, y);
    if (a.w_post) {
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
            for (int k = 0; k < VE; ++k)
                s += y[u][k] * y[u][k];
        block_sums<1>(&s, lds, turn);
        const float p = 1.0f / __builtin_sqrtf(s * a.inv_hidden + a.eps);
        if (a.rstd_post && tid == 0)
            a.rstd_post[t] = p;
        if (!kAhead) load(wpost, a.w_post);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float w[VE];
            unpack<DT>(fixed<DT, TAIL>(wpost[u], tid + u * bd, hidden), w);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                y[u][k] = y[u][k] * p * w[k];
        }
    }
    if (grow) {
        if (!kAhead) load(gv, grow);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float g[VE];
            unpack<DT>(fixed<DT, TAIL>(gv[u], tid + u * bd, hidden), g);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                y[u][k] *= g[k];
        }
    }
    if (a.residual) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float f[VE];
            unpack<DT>(fixed<DT, TAIL>(res[u], tid + u * bd, hidden), f);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                y[u][k] += a.residual_scale * f[k];
        }
    }
    if (a.out_h) {
#pragma unroll
        for (int u = 0; u < NV; ++u)
            st_row<DT, TAIL, true>(static_cast<char*>(a.out_h) + t * a.ld_h * EB, tid + u * bd, hidden, pack<DT>(y[u]));
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
    if (a.rstd_pre && tid == 0)
        a.rstd_pre[t] = q;
    if (!kAhead) load(wpre, a.w_pre);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float w[VE];
        unpack<DT>(fixed<DT, TAIL>(wpre[u], tid + u * bd, hidden), w);
#pragma unroll
        for (int k = 0; k < VE; ++k)
            w[k] = y[u][k] * q * w[k];
        st_row<DT, TAIL, true>(static_cast<char*>(a.out_z) + t * a.ld_z * EB, tid + u * bd, hidden, pack<DT>(w));
    }
}

template <int NV, int WG>
const void* norm_of(int dtype, bool tail)
{
    if (dtype == 0)
        return tail ? (const void*)k_norm<0, true, NV, WG> : (const void*)k_norm<0, false, NV, WG>;
    return tail ? (const void*)k_norm<1, true, NV, WG> : (const void*)k_norm<1, false, NV, WG>;
}
const void* norm_fn(int dtype, bool tail, unsigned wg, size_t nvec)
{
    const size_t nv = (nvec + wg - 1) / wg;
    if (wg <= 256)
        return nv <= 1 ? norm_of<1, 256>(dtype, tail) : norm_of<2, 256>(dtype, tail);
    return nv <= 1   ? norm_of<1, 1024>(dtype, tail)
           : nv <= 2 ? norm_of<2, 1024>(dtype, tail)
           : nv <= 4 ? norm_of<4, 1024>(dtype, tail)
                     : norm_of<8, 1024>(dtype, tail);
}

// Two vectors a thread where up to 1024 threads allow it; one where there are
// no more rows than CUs, for the latency. Whole waves only: a row of 1251
// vectors takes 640 threads, three to a CU.
unsigned norm_threads(size_t nvec, size_t rows)
{
    const size_t per = rows <= (size_t)device_cu_count() ? 1 : 2, t = (nvec + per - 1) / per;
    return t >= 1024 ? 1024u : t < kWave ? (unsigned)kWave : (unsigned)((t + kWave - 1) / kWave * kWave);
}

}  // namespace

hipError_t launch_norm(const NormArgs& in, int dtype, hipStream_t s)
{
    NormArgs a = in;
    void* params[] = {&a};
    const size_t nvec = vectors(a.hidden, dtype);
    const unsigned wg = norm_threads(nvec, a.rows);
    return launch_logged("k_norm", norm_fn(dtype, partial(a.hidden, dtype), wg, nvec), dim3((unsigned)a.rows), dim3(wg),
                         params, s);
}

}  // namespace rx
