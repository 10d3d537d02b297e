// philox.hpp -- the generator of dropout's mask: Philox of four words and ten
// rounds (J. Salmon, M. Moraes, R. Dror, D. Shaw: "Parallel random numbers: as
// easy as 1, 2, 3", 2011). A number of it depends on its counter and the key
// alone, so the backward pass makes the forward's mask again.
#pragma once

#include "block_common.hpp"

namespace rx {
namespace {

// Which elements of a call are dropped, as its kernels know it.
struct Dropper {
    uint64_t seed, offset;
    uint64_t first;        // the row's first counter
    uint32_t threshold;    // 65536 p
};

__device__ __forceinline__ u32x4 philox(uint64_t i, const Dropper& d)
{
    uint32_t c0 = (uint32_t)i, c1 = (uint32_t)(i >> 32), c2 = (uint32_t)d.offset, c3 = (uint32_t)(d.offset >> 32);
    uint32_t k0 = (uint32_t)d.seed, k1 = (uint32_t)(d.seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = (uint64_t)0xD2511F53u * c0, q = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)q;
        c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// f of vector v of the row: multiplied with `gain` where it is kept, 0 where
// it is dropped. 16 bits an element: a number of the generator makes a vector
// of BF16, or two of FP32.
template <int DT>
__device__ __forceinline__ void drop_vector(const Dropper& d, int v, float gain, float* f)
{
    const u32x4 x = philox(d.first + (uint32_t)(DT == 0 ? v >> 1 : v), d);
    uint32_t w[Elem<DT>::kVE / 2];
    if constexpr (DT == 0) {
        w[0] = v & 1 ? x[2] : x[0];
        w[1] = v & 1 ? x[3] : x[1];
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = x[k];
    }
#pragma unroll
    for (int k = 0; k < Elem<DT>::kVE; ++k) {
        const uint32_t half = k & 1 ? w[k / 2] >> 16 : w[k / 2] & 0xFFFFu;
        f[k] = half >= d.threshold ? f[k] * gain : 0.0f;
    }
}

}  // namespace
}  // namespace rx
