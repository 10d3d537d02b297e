// gemm_fp4.hip -- rows to 4-bit floating point with a scale for each group, and
// the choice of the product's translation unit (gfx950). Defined in rx.h.
#include "block_common.hpp"

namespace rx {
namespace {

// A group's scale and multiplier from its absmax A, as i8_scale() with 6 for 127.
__device__ __forceinline__ void fp4_scale(float a, float& s, float& r)
{
    const float sv = a / 6.0f, rv = 6.0f / a;
    const bool degenerate = (a == 0.0f) | (sv == 0.0f) | !__builtin_isfinite(rv);
    const bool finite = __builtin_isfinite(a);
    s = !finite ? a : degenerate ? 1.0f : sv;
    r = !finite ? 0.0f : degenerate ? 1.0f : rv;
}

// A workgroup a row, a lane a vector: 4 to 32 neighbouring lanes have a group. 8192 x 8192
// takes 59 us in FP32 (5.2 TB/s), which the bytes bound, and 43 in BF16 (4.0): there a thread's
// four loads, each waited for by its group's maximum before the next goes out (waves
// wait 72% of their cycles). Once for weights that are then multiplied many times.
template <int DT, bool TAIL>
__global__ __launch_bounds__(256) void k_quant_fp4(QuantFp4Args a)
{
    constexpr int VE = Elem<DT>::kVE;
    const size_t t = blockIdx.x;
    const int k = (int)a.k, nvec = (k + VE - 1) / VE, lanes = a.group / VE;
    const size_t groups = (a.k + a.group - 1) / a.group;
    const void* row = static_cast<const char*>(a.x) + t * a.ld_x * Elem<DT>::kBytes;
    for (int v0 = 0; v0 < nvec; v0 += (int)blockDim.x) {
        const int v = v0 + (int)threadIdx.x;
        const u32x4 x = ld_row<DT, TAIL, true>(row, v < nvec ? v : nvec - 1, k);
        float s, r;
        fp4_scale(bits_f32(group_max_rt(v < nvec ? vec_absmax<DT>(x) : 0, lanes)), s, r);
        if (v >= nvec)
            continue;
        if (v % lanes == 0)
            a.scales[t * groups + v / lanes] = s;
        float f[VE];
        unpack<DT>(x, f);
        uint32_t q = 0;
#pragma unroll
        for (int i = 0; i < VE; ++i)
            f[i] = r == 0.0f ? 0.0f : f[i] * r;   // a NaN's product has no code
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[0], f[1], 1.0f, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[2], f[3], 1.0f, 1);
        if constexpr (VE == 8) {
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[4], f[5], 1.0f, 2);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[6], f[7], 1.0f, 3);
        }
        uint8_t* p = a.codes + t * a.ld_codes + (size_t)v * (VE / 2);
        const int left = k - v * VE;
        if (!TAIL || left >= VE) {
            if constexpr (VE == 8)
                *reinterpret_cast<u32_any*>(p) = q;
            else
                *reinterpret_cast<u16_any*>(p) = (uint16_t)q;
        } else {
            for (int b = 0; b < (left + 1) / 2; ++b)
                p[b] = (uint8_t)(q >> (8 * b));
        }
    }
}

}  // namespace

hipError_t launch_quant_fp4(const QuantFp4Args& in, int dtype, hipStream_t s)
{
    QuantFp4Args a = in;
    void* params[] = {&a};
    const bool tail = partial(a.k, dtype);
    const void* fn = dtype == 0 ? tail ? (const void*)k_quant_fp4<0, true> : (const void*)k_quant_fp4<0, false>
                     : tail     ? (const void*)k_quant_fp4<1, true>
                                : (const void*)k_quant_fp4<1, false>;
    return launch_logged("k_quant_fp4", fn, dim3((unsigned)a.rows), dim3(threads_for(vectors(a.k, dtype), 256)), params, s);
}

hipError_t launch_gemm_fp4(const GemmFp4Args& a, int dtype, hipStream_t s)
{
    if (dtype == 0)
        return a.group == 32 ? launch_fp4_fp32_32(a, s) : a.group == 64 ? launch_fp4_fp32_64(a, s) : launch_fp4_fp32_128(a, s);
    return a.group == 32 ? launch_fp4_bf16_32(a, s) : a.group == 64 ? launch_fp4_bf16_64(a, s) : launch_fp4_bf16_128(a, s);
}

}  // namespace rx
