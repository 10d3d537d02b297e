// norm_common.hpp -- what the norms and their gradients share (norm.hip,
// norm_backward.hip, layer_norm.hip).
#pragma once

#include "block_common.hpp"

namespace rx {
namespace {

// Sums of c[0 .. N) over the NW waves that hold a row, the same in every
// thread (NW 0: over the workgroup's). `lds` holds 2 x 16 x N floats, used in
// halves by turns, so one barrier a call is enough: a half is written again
// only after the next call's barrier.
template <int N, int NW = 0>
__device__ __forceinline__ void block_sums(float* c, float* lds, int& turn)
{
    const int nw = NW ? NW : blockDim.x / kWave;
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
// Thread `tid` of the `threads` that hold the row has vectors tid + u threads.
template <int DT, bool TAIL, int NV, int B, bool FIRST>
__device__ __forceinline__ void fold_batch(const void* const* src, int r, size_t row_bytes, int hidden, int tid,
                                           int threads, float (*y)[Elem<DT>::kVE])
{
    constexpr int VE = Elem<DT>::kVE;
    u32x4 x[B][NV];
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
        for (int u = 0; u < NV; ++u)
            x[b][u] = ld_raw<DT, TAIL, true>(static_cast<const char*>(src[r + b]) + row_bytes, tid + u * threads, hidden);
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float f[VE];
            unpack<DT>(fixed<DT, TAIL>(x[b][u], tid + u * threads, hidden), f);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                y[u][k] = FIRST && b == 0 ? f[k] : y[u][k] + f[k];
        }
}

// y = the sources' sum in their order, B sources' loads of a thread in flight
// together; thread `tid` of the `bd` that hold the row.
template <int DT, bool TAIL, int NV>
__device__ __forceinline__ void fold_row(const void* const* src, int nsrc, size_t row_bytes, int hidden, int tid, int bd,
                                         float (*y)[Elem<DT>::kVE])
{
    constexpr int VE = Elem<DT>::kVE, B = NV == 1 ? 8 : 4;   // more would cost a longer row its occupancy
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

}  // namespace
}  // namespace rx
