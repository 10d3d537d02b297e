// norm.hip -- the sum over the ranks fused with the norms, the gate and the
// residual around a block (gfx950). Defined in rx.h.
//
// One workgroup holds a row in registers, so every input is read once and
// every output written once: the sums for the two norms are the only thing
// that crosses lanes. HBM-bound (a few flops a byte).
#include "norm_common.hpp"

namespace rx {
namespace {

template <int DT, bool TAIL, int NV>
__device__ __forceinline__ void fold_row(const void* const* src, int nsrc, size_t row_bytes, int hidden,
                                         float (*y)[Elem<DT>::kVE])
{
    int r;
    switch (nsrc) {
    case 1: fold_batch<DT, TAIL, NV, 1, true>(src, 0, row_bytes, hidden, (int)threadIdx.x, (int)blockDim.x, y); return;
    case 2: fold_batch<DT, TAIL, NV, 2, true>(src, 0, row_bytes, hidden, (int)threadIdx.x, (int)blockDim.x, y); return;
    case 3: fold_batch<DT, TAIL, NV, 3, true>(src, 0, row_bytes, hidden, (int)threadIdx.x, (int)blockDim.x, y); return;
    default: fold_batch<DT, TAIL, NV, 4, true>(src, 0, row_bytes, hidden, (int)threadIdx.x, (int)blockDim.x, y); r = 4;
    }
    for (; r + 4 <= nsrc; r += 4)
        fold_batch<DT, TAIL, NV, 4, false>(src, r, row_bytes, hidden, (int)threadIdx.x, (int)blockDim.x, y);
    for (; r < nsrc; ++r)
        fold_batch<DT, TAIL, NV, 1, false>(src, r, row_bytes, hidden, (int)threadIdx.x, (int)blockDim.x, y);
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

// Two vectors a thread where up to 1024 threads allow it.
unsigned norm_threads(size_t nvec) { return threads_for((nvec + 1) / 2, 1024); }

}  // namespace

hipError_t launch_norm(const NormArgs& in, int dtype, hipStream_t s)
{
    NormArgs a = in;
    void* params[] = {&a};
    const size_t nvec = vectors(a.hidden, dtype);
    const unsigned wg = norm_threads(nvec);
    return launch_logged("k_norm", norm_fn(dtype, partial(a.hidden, dtype), wg, nvec), dim3((unsigned)a.rows), dim3(wg),
                         params, s);
}

}  // namespace rx
