// block_common.hpp -- helpers of the operators around a block's allreduce
// (moe.hip, norm.hip, gemm_i8.hip): rows of any length and alignment in
// 16-byte vectors, and sums across a wave or a workgroup.
#pragma once

#include <type_traits>

#include "rx_device.hpp"
#include "rx_internal.hpp"

namespace rx {
namespace {

template <int DT> struct Elem;
template <> struct Elem<0> { static constexpr int kVE = 4, kBytes = 4; };  // FP32
template <> struct Elem<1> { static constexpr int kVE = 8, kBytes = 2; };  // BF16

// 16 bytes at the alignment of one element: the vector memory instructions
// take any address, so rows of odd length need no kernel of their own.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));

__device__ __forceinline__ u32x4 ld16_any(const void* p)
{
    return *reinterpret_cast<const u32x4_any*>(p);
}
__device__ __forceinline__ u32x4 ld16_any_stream(const void* p)
{
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
}
__device__ __forceinline__ void st16_any(void* p, u32x4 v)
{
    *reinterpret_cast<u32x4_any*>(p) = v;
}
__device__ __forceinline__ void st16_any_stream(void* p, u32x4 v)
{
    __builtin_nontemporal_store((u32x4_any)v, reinterpret_cast<u32x4_any*>(p));
}

// Vector v of a row of `hidden` elements. TAIL: the row's last vector may be
// partial (its missing elements read as 0 and are not written); vectors past
// the row are 0. Without TAIL hidden is a multiple of the vector. A row is
// shorter than 2^32 bytes: with a uniform row pointer the 32-bit offset lets
// the address stay in scalar registers.
//
// A partial vector is the last whole one of the row, shifted: one load, where
// one for every element would be a chain of up to seven. ld_raw loads and
// fixed() shifts: between the two go the other loads, so that none waits.
// Without SHORT a row is a vector long at least: the code for shorter ones
// writes the same registers element by element, and a load in a loop would wait for
// the one before it.
template <int DT, bool TAIL, bool NT = false, bool SHORT = true>
__device__ __forceinline__ u32x4 ld_raw(const void* row, int v, int hidden)
{
    constexpr int VE = Elem<DT>::kVE;
    const int c = v * VE;
    const char* p = static_cast<const char*>(row);
    u32x4 x = {0, 0, 0, 0};
    if (!TAIL || !SHORT || hidden >= VE) {
        const int at = !TAIL || c < hidden - VE ? c : hidden - VE;
        if (TAIL || c < hidden) {
            p += (uint32_t)at * (uint32_t)Elem<DT>::kBytes;
            x = NT ? ld16_any_stream(p) : ld16_any(p);
        }
    } else if (c < hidden) {   // a row shorter than a vector
#pragma unroll
        for (int e = 0; e < VE - 1; ++e)
            if (e < hidden) {
                if constexpr (DT == 0)
                    x[e] = reinterpret_cast<const uint32_t*>(p)[e];
                else
                    x[e / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[e] << (16 * (e & 1));
            }
    }
    return x;
}

template <int DT, bool TAIL>
__device__ __forceinline__ u32x4 fixed(u32x4 x, int v, int hidden)
{
    constexpr int VE = Elem<DT>::kVE;
    const int d = v * VE + VE - hidden;   // elements past the row
    if (TAIL && d > 0 && hidden >= VE) {
        const uint64_t lo = x[0] | (uint64_t)x[1] << 32, hi = x[2] | (uint64_t)x[3] << 32;
        const int s = d * Elem<DT>::kBytes * 8;   // bits
        const uint64_t l = s < 64 ? lo >> s | hi << (64 - s) : s < 128 ? hi >> (s - 64) : 0;
        const uint64_t h = s < 64 ? hi >> s : 0;
        x = u32x4{(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)h, (uint32_t)(h >> 32)};
    }
    return x;
}

template <int DT, bool TAIL, bool NT = false>
__device__ __forceinline__ u32x4 ld_row(const void* row, int v, int hidden)
{
    return fixed<DT, TAIL>(ld_raw<DT, TAIL, NT>(row, v, hidden), v, hidden);
}

template <int DT, bool TAIL, bool NT = false>
__device__ __forceinline__ void st_row(void* row, int v, int hidden, u32x4 x)
{
    constexpr int VE = Elem<DT>::kVE;
    const int c = v * VE;
    char* p = static_cast<char*>(row) + (uint32_t)c * (uint32_t)Elem<DT>::kBytes;
    if (!TAIL || c + VE <= hidden) {
        if (TAIL || c < hidden) {
            if (NT) st16_any_stream(p, x); else st16_any(p, x);
        }
    } else if (c < hidden) {
        const int n = (hidden - c) * Elem<DT>::kBytes;   // bytes
        if (n & 8) {
            *reinterpret_cast<u32x2_any*>(p) = (u32x2_any){x[0], x[1]};
            x[0] = x[2];
            x[1] = x[3];
            p += 8;
        }
        if (n & 4) {
            *reinterpret_cast<u32_any*>(p) = x[0];
            x[0] = x[1];
            p += 4;
        }
        if (DT != 0 && (n & 2))
            *reinterpret_cast<uint16_t*>(p) = (uint16_t)x[0];
    }
}

template <int DT>
__device__ __forceinline__ void unpack(u32x4 x, float* f)
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == 0) {
            f[k] = bits_f32(x[k]);
        } else {
            f[2 * k] = bf16_lo(x[k]);
            f[2 * k + 1] = bf16_hi(x[k]);
        }
    }
}

template <int DT>
__device__ __forceinline__ u32x4 pack(const float* f)
{
    u32x4 x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == 0)
            x[k] = __builtin_bit_cast(uint32_t, f[k]);
        else
            x[k] = pack_bf16(f[2 * k], f[2 * k + 1]);
    }
    return x;
}

// Sum over the wave, the same in every lane (and the same bits: each step
// adds a lane and its mirror, and FP32 addition commutes).
__device__ __forceinline__ float wave_sum(float v)
{
    auto u = [](float x) { return __builtin_bit_cast(uint32_t, x); };
    v += bits_f32(dpp<0xB1>(u(v)));
    v += bits_f32(dpp<0x4E>(u(v)));
    v += bits_f32(dpp<0x141>(u(v)));
    v += bits_f32(dpp<0x140>(u(v)));
    auto p = __builtin_amdgcn_permlane16_swap(u(v), u(v), false, false);
    v = bits_f32(p[0]) + bits_f32(p[1]);
    auto q = __builtin_amdgcn_permlane32_swap(u(v), u(v), false, false);
    return bits_f32(q[0]) + bits_f32(q[1]);
}

__device__ __forceinline__ uint32_t wave_sum_u(uint32_t v)
{
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = p[0] + p[1];
    auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return q[0] + q[1];
}

// Sum over aligned groups of G lanes, the same in each of them.
template <int G>
__device__ __forceinline__ float group_sum(float v)
{
    auto u = [](float x) { return __builtin_bit_cast(uint32_t, x); };
    if constexpr (G >= 2) v += bits_f32(dpp<0xB1>(u(v)));
    if constexpr (G >= 4) v += bits_f32(dpp<0x4E>(u(v)));
    if constexpr (G >= 8) v += bits_f32(dpp<0x141>(u(v)));
    if constexpr (G >= 16) v += bits_f32(dpp<0x140>(u(v)));
    if constexpr (G >= 32) {
        auto p = __builtin_amdgcn_permlane16_swap(u(v), u(v), false, false);
        v = bits_f32(p[0]) + bits_f32(p[1]);
    }
    if constexpr (G >= 64) {
        auto p = __builtin_amdgcn_permlane32_swap(u(v), u(v), false, false);
        v = bits_f32(p[0]) + bits_f32(p[1]);
    }
    return v;
}

// ... of a number of lanes that is the same for the wave.
__device__ __forceinline__ float group_sum_rt(float v, int g)
{
    auto u = [](float x) { return __builtin_bit_cast(uint32_t, x); };
    if (g >= 2) v += bits_f32(dpp<0xB1>(u(v)));
    if (g >= 4) v += bits_f32(dpp<0x4E>(u(v)));
    if (g >= 8) v += bits_f32(dpp<0x141>(u(v)));
    if (g >= 16) v += bits_f32(dpp<0x140>(u(v)));
    if (g >= 32) {
        auto p = __builtin_amdgcn_permlane16_swap(u(v), u(v), false, false);
        v = bits_f32(p[0]) + bits_f32(p[1]);
    }
    if (g >= 64) {
        auto p = __builtin_amdgcn_permlane32_swap(u(v), u(v), false, false);
        v = bits_f32(p[0]) + bits_f32(p[1]);
    }
    return v;
}

// Sum over the lanes at this one's place in each group of G, the same in all.
template <int G>
__device__ __forceinline__ float across(float v)
{
    auto u = [](float x) { return __builtin_bit_cast(uint32_t, x); };
    if constexpr (G <= 1) v += bits_f32(dpp<0x121>(u(v)));   // row_ror 1, 2, 4, 8
    if constexpr (G <= 2) v += bits_f32(dpp<0x122>(u(v)));
    if constexpr (G <= 4) v += bits_f32(dpp<0x124>(u(v)));
    if constexpr (G <= 8) v += bits_f32(dpp<0x128>(u(v)));
    if constexpr (G <= 16) {
        auto p = __builtin_amdgcn_permlane16_swap(u(v), u(v), false, false);
        v = bits_f32(p[0]) + bits_f32(p[1]);
    }
    if constexpr (G <= 32) {
        auto p = __builtin_amdgcn_permlane32_swap(u(v), u(v), false, false);
        v = bits_f32(p[0]) + bits_f32(p[1]);
    }
    return v;
}
template <int G>
__device__ __forceinline__ uint32_t across(uint32_t v)
{
    if constexpr (G <= 1) v += dpp<0x121>(v);
    if constexpr (G <= 2) v += dpp<0x122>(v);
    if constexpr (G <= 4) v += dpp<0x124>(v);
    if constexpr (G <= 8) v += dpp<0x128>(v);
    if constexpr (G <= 16) {
        auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = p[0] + p[1];
    }
    if constexpr (G <= 32) {
        auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = p[0] + p[1];
    }
    return v;
}

// ... of a number of lanes that is the same for the wave.
__device__ __forceinline__ float across_rt(float v, int g)
{
    auto u = [](float x) { return __builtin_bit_cast(uint32_t, x); };
    if (g <= 1) v += bits_f32(dpp<0x121>(u(v)));
    if (g <= 2) v += bits_f32(dpp<0x122>(u(v)));
    if (g <= 4) v += bits_f32(dpp<0x124>(u(v)));
    if (g <= 8) v += bits_f32(dpp<0x128>(u(v)));
    if (g <= 16) {
        auto p = __builtin_amdgcn_permlane16_swap(u(v), u(v), false, false);
        v = bits_f32(p[0]) + bits_f32(p[1]);
    }
    if (g <= 32) {
        auto p = __builtin_amdgcn_permlane32_swap(u(v), u(v), false, false);
        v = bits_f32(p[0]) + bits_f32(p[1]);
    }
    return v;
}

// What the wave's lanes wrote to LDS is there for all of them: its LDS
// instructions run in order, so only the compiler has to keep theirs.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Inclusive sum over the lanes up to this one.
__device__ __forceinline__ uint32_t wave_incl(uint32_t v)
{
    auto from = [](uint32_t x, auto ctrl, auto rows) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl(), rows(), 0xF, false);
    };
    using std::integral_constant;
    v += from(v, integral_constant<int, 0x111>(), integral_constant<int, 0xF>());   // one lane up within 16
    v += from(v, integral_constant<int, 0x112>(), integral_constant<int, 0xF>());
    v += from(v, integral_constant<int, 0x114>(), integral_constant<int, 0xF>());
    v += from(v, integral_constant<int, 0x118>(), integral_constant<int, 0xF>());
    v += from(v, integral_constant<int, 0x142>(), integral_constant<int, 0xA>());   // lane 15 of a row to the next row
    v += from(v, integral_constant<int, 0x143>(), integral_constant<int, 0xC>());   // lane 31 to the upper half
    return v;
}

// The largest magnitude of a vector, as bits.
template <int DT>
__device__ __forceinline__ uint32_t vec_absmax(u32x4 x)
{
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == 0)
            m = umax(m, x[k] & 0x7FFFFFFFu);
        else
            m = umax(m, umax((x[k] << 16) & 0x7FFFFFFFu, x[k] & 0x7FFF0000u));
    }
    return m;
}

// A row's INT8 scale and multiplier from its absmax A: fl32(A / 127) and
// fl32(127 / A); 1 where a quotient is useless, A and 0 where A is not finite
// (its products are then NaN). Once a row: plain divisions.
__device__ __forceinline__ void i8_scale(float a, float& s, float& r)
{
    const float sv = a / 127.0f, rv = 127.0f / a;
    const bool degenerate = (a == 0.0f) | (sv == 0.0f) | !__builtin_isfinite(rv);
    const bool finite = __builtin_isfinite(a);
    s = !finite ? a : degenerate ? 1.0f : sv;
    r = !finite ? 0.0f : degenerate ? 1.0f : rv;
}

// The codes of a vector, 4 a word. |x r| <= 127 (1 + 2^-23), so adding
// 1.5 2^23 rounds to the nearest integer, ties to even, and leaves its two's
// complement in the sum's low byte.
template <int DT>
__device__ __forceinline__ void i8_codes(u32x4 x, float r, uint32_t* q)
{
    constexpr int VE = Elem<DT>::kVE;
    float f[VE];
    unpack<DT>(x, f);
    uint32_t b[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k)
        b[k] = __builtin_bit_cast(uint32_t, f[k] * r + 12582912.0f);
#pragma unroll
    for (int k = 0; k < VE / 4; ++k) {
        const uint32_t lo = __builtin_amdgcn_perm(b[4 * k + 1], b[4 * k], 0x0C0C0400);      // bytes 0, 0
        const uint32_t hi = __builtin_amdgcn_perm(b[4 * k + 3], b[4 * k + 2], 0x0C0C0400);
        q[k] = r == 0.0f ? 0 : lo | hi << 16;   // a NaN's product may have any low byte
    }
}

// Vector v's codes into a row of `hidden` bytes.
template <int DT, bool TAIL>
__device__ __forceinline__ void st_codes(void* row, int v, int hidden, const uint32_t* q)
{
    constexpr int VE = Elem<DT>::kVE;
    const int c = v * VE;
    uint8_t* p = static_cast<uint8_t*>(row) + c;
    if (!TAIL || c + VE <= hidden) {
        if (TAIL || c < hidden) {
            if constexpr (VE == 8)
                *reinterpret_cast<u32x2_any*>(p) = (u32x2_any){q[0], q[1]};
            else
                *reinterpret_cast<u32_any*>(p) = q[0];
        }
    } else if (c < hidden) {
        const int n = hidden - c;
        uint32_t w = q[0];
        if (VE == 8 && (n & 4)) {
            *reinterpret_cast<u32_any*>(p) = w;
            w = q[VE / 4 - 1];
            p += 4;
        }
        if (n & 2) {
            *reinterpret_cast<u16_any*>(p) = (uint16_t)w;
            w >>= 16;
            p += 2;
        }
        if (n & 1)
            *p = (uint8_t)w;
    }
}

// 64 to `most` threads, at least one for each vector where that is enough.
inline unsigned threads_for(size_t nvec, unsigned most)
{
    unsigned t = 64;
    while (t < most && t < nvec)
        t *= 2;
    return t;
}
inline size_t vectors(size_t hidden, int dtype) { return (hidden + (dtype ? 7 : 3)) / (dtype ? 8 : 4); }
inline bool partial(size_t hidden, int dtype) { return hidden % (dtype ? 8 : 4) != 0; }

}  // namespace
}  // namespace rx
