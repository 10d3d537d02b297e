// route.hip -- each token's experts from the router's logits, the counts and
// the losses over all tokens, and their gradient (gfx950). Defined in rx.h.
//
// G lanes hold a token's logits, V neighbouring ones each, and a wave 64 / G
// tokens: a maximum over a token costs log2 G steps between lanes and V / 2
// within one, so few lanes with many logits each are cheaper than a wave a
// token. A lane keeps the same experts for all its tokens, so the sums over
// the tokens stay in its registers and meet in LDS at the end.
#include "block_common.hpp"

namespace rx {
namespace {

constexpr int kRouteWaves = 4;

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

// Logits pos V .. pos V + V - 1 of a row.
template <int DT, int V>
__device__ __forceinline__ void ld_logits(const void* row, int pos, int experts, float* x)
{
    constexpr int VE = Elem<DT>::kVE;
    u32x4 r[V / VE];
#pragma unroll
    for (int i = 0; i < V / VE; ++i)
        r[i] = ld_raw<DT, true>(row, pos * (V / VE) + i, experts);
#pragma unroll
    for (int i = 0; i < V / VE; ++i)
        unpack<DT>(fixed<DT, true>(r[i], pos * (V / VE) + i, experts), x + i * VE);
}

// Unsigned numbers in the logits' order: -inf is kKeyNone, what is taken or
// past the experts 0, NaN above all; -0 equals 0.
constexpr uint32_t kKeyNone = 0x007FFFFFu;
__device__ __forceinline__ uint32_t key_of(float x)
{
    uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
    u = x != x ? 0x7FC00000u : u;
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key)
{
    return bits_f32(key ^ (key >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

// What a workgroup leaves for the second launch: experts counts, experts sums
// of P, its tokens and the sum of their lse^2.
__device__ __forceinline__ uint32_t part_words(int experts) { return 2 * (uint32_t)experts + 2; }

template <int DT, int G, int V, bool SUMS>
__global__ __launch_bounds__(kRouteWaves * kWave) void k_route(RouteArgs a)
{
    constexpr int TW = kWave / G;                                // tokens of a wave
    constexpr int MOST = V * G < kMaxTopk ? V * G : kMaxTopk;    // choices of a token
    struct Pick {
        int id;
        float e;
    };
    __shared__ Pick picks[kRouteWaves][TW * MOST];
    __shared__ uint32_t sums[SUMS ? kRouteWaves : 1][SUMS ? V * G : 1];
    __shared__ uint32_t totals[kRouteWaves][2];
    const int lane = lane_id(), wave = threadIdx.x / kWave, pos = lane % G, sub = lane / G;
    const int experts = a.experts, topk = a.topk;
    float prob[V] = {}, squares = 0.0f;
    uint32_t count[V] = {}, live_tokens = 0;
    const size_t step = (size_t)gridDim.x * kRouteWaves * TW;
    for (size_t t0 = ((size_t)blockIdx.x * kRouteWaves + wave) * TW; t0 < a.tokens; t0 += step) {
        const size_t t = t0 + sub;
        bool live = t < a.tokens && (!a.mask || a.mask[t]);
        float x[V];
        uint32_t key[V];
        if (live)
            ld_logits<DT, V>(static_cast<const char*>(a.logits) + t * a.ld * Elem<DT>::kBytes, pos, experts, x);
#pragma unroll
        for (int i = 0; i < V; ++i)
            key[i] = live && pos * V + i < experts ? key_of(x[i]) : 0;
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            mine = umax(mine, key[i]);
        uint32_t top = group_max<G>(mine);
        live = top > kKeyNone;
        const float high = live ? value_of(top) : 0.0f;
        float sum = 0.0f, e[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            e[i] = live && pos * V + i < experts ? expf(x[i] - high) : 0.0f;
            sum += e[i];
        }
        sum = group_sum<G>(sum);
        // the choices, one a round
        Pick* pick = picks[wave] + sub * topk;
        float chosen = 0.0f;
        uint32_t taken = 0;
        for (int j = 0; j < topk; ++j) {
            const uint64_t owners = __ballot(mine == top) >> (sub * G);
            const bool any = top > kKeyNone, owner = any && pos == __builtin_ctzll(owners);
            const float w = any ? expf(value_of(top) - high) : 0.0f;
            chosen += w;
            if (owner) {
                uint32_t first = 0;
#pragma unroll
                for (int i = V - 1; i >= 0; --i)
                    first = key[i] == top ? (uint32_t)i : first;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    key[i] = (uint32_t)i == first ? 0 : key[i];
                taken |= 1u << first;
                pick[j] = Pick{pos * V + (int)first, w};
                mine = 0;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    mine = umax(mine, key[i]);
            }
            if (!any && pos == 0)
                pick[j] = Pick{-1, 0.0f};
            top = group_max<G>(mine);
        }
        const float by = a.renormalize ? chosen : sum;
        const float scale = live ? by : 1.0f;
        if (a.lse && pos == 0 && t < a.tokens)
            a.lse[t] = live ? high + logf(sum) : -__builtin_inff();
        // tokens of the wave follow each other: their choices too
        const size_t left = a.tokens - t0;
        const int n = (left < (size_t)TW ? (int)left : TW) * topk;
        wave_sync();
        for (int i0 = 0; i0 < n; i0 += kWave) {
            const int i = i0 + lane;
            // the divisor of the token that choice i belongs to
            const float div = bits_f32((uint32_t)__builtin_amdgcn_ds_bpermute((i < n ? i / topk : 0) * G * 4, (int)__builtin_bit_cast(uint32_t, scale)));
            if (i < n) {
                const Pick p = picks[wave][i];
                a.ids[t0 * topk + i] = p.id;
                a.weights[t0 * topk + i] = p.e / div;
            }
        }
        wave_sync();
        if constexpr (SUMS) {
            const float inv = 1.0f / (live ? sum : 1.0f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                prob[i] += e[i] * inv;
                count[i] += taken >> i & 1;
            }
            if (live && pos == 0) {
                const float l = high + logf(sum);
                squares += l * l;
                ++live_tokens;
            }
        }
    }
    if constexpr (SUMS) {
        // over the wave's groups, then over the waves, in their order
        uint32_t* out = a.workspace + 1 + (size_t)blockIdx.x * part_words(experts);
        auto across = [&](float v) {
            for (int d = G; d < kWave; d *= 2)
                v += bits_f32((uint32_t)__builtin_amdgcn_ds_bpermute((lane ^ d) * 4, (int)__builtin_bit_cast(uint32_t, v)));
            return v;
        };
        auto across_u = [&](uint32_t v) {
            for (int d = G; d < kWave; d *= 2)
                v += (uint32_t)__builtin_amdgcn_ds_bpermute((lane ^ d) * 4, (int)v);
            return v;
        };
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c = across_u(count[i]);
            if (sub == 0)
                sums[wave][pos * V + i] = c;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < experts; e += kRouteWaves * kWave) {
            uint32_t c = 0;
            for (int w = 0; w < kRouteWaves; ++w)
                c += sums[w][e];
            out[e] = c;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float p = across(prob[i]);
            if (sub == 0)
                sums[wave][pos * V + i] = __builtin_bit_cast(uint32_t, p);
        }
        squares = wave_sum(squares);
        live_tokens = wave_sum_u(live_tokens);
        if (lane == 0) {
            totals[wave][0] = live_tokens;
            totals[wave][1] = __builtin_bit_cast(uint32_t, squares);
        }
        __syncthreads();
        for (int e = threadIdx.x; e < experts; e += kRouteWaves * kWave) {
            float p = 0.0f;
            for (int w = 0; w < kRouteWaves; ++w)
                p += bits_f32(sums[w][e]);
            out[experts + e] = __builtin_bit_cast(uint32_t, p);
        }
        if (threadIdx.x == 0) {
            uint32_t n = 0;
            float z = 0.0f;
            for (int w = 0; w < kRouteWaves; ++w) {
                n += totals[w][0];
                z += bits_f32(totals[w][1]);
            }
            out[2 * experts] = n;
            out[2 * experts + 1] = __builtin_bit_cast(uint32_t, z);
        }
    }
}

// The workgroups' sums in their order, and the losses: one workgroup.
__global__ __launch_bounds__(1024) void k_route_sums(RouteArgs a)
{
    __shared__ float lds[16];
    __shared__ uint32_t lds_n[16];
    __shared__ float lds_z[16];
    const int experts = a.experts, lane = lane_id(), wave = threadIdx.x / kWave;
    const uint32_t* in = a.workspace + 1;
    const size_t words = part_words(experts);
    float dot = 0.0f;
    for (int e = threadIdx.x; e < experts; e += 1024) {
        uint32_t c = 0;
        float p = 0.0f;
        for (uint32_t g = 0; g < a.parts; ++g) {
            c += in[g * words + e];
            p += bits_f32(in[g * words + experts + e]);
        }
        a.counts[e] = (int)c;
        dot += (float)c * p;
    }
    uint32_t n = 0;
    float z = 0.0f;
    for (uint32_t g = threadIdx.x; g < a.parts; g += 1024) {
        n += in[g * words + 2 * experts];
        z += bits_f32(in[g * words + 2 * experts + 1]);
    }
    n = wave_sum_u(n);
    z = wave_sum(z);
    dot = wave_sum(dot);
    if (lane == 0) {
        lds[wave] = dot;
        lds_n[wave] = n;
        lds_z[wave] = z;
    }
    __syncthreads();
    if (threadIdx.x)
        return;
    dot = z = 0.0f;
    n = 0;
    for (int w = 0; w < 16; ++w) {
        dot += lds[w];
        n += lds_n[w];
        z += lds_z[w];
    }
    a.counts[experts] = (int)n;
    const float inv = n ? 1.0f / (float)n : 0.0f;
    a.losses[0] = dot * inv * inv * ((float)experts / (float)a.topk);
    a.losses[1] = z * inv;
}

// ---- gradient ------------------------------------------------------------------

// dl = P (c f + h - A + z), with c f from the counts, h and A from the weights'
// gradients: an element of the token's choices in LDS at a time.
template <int DT, int G, int V>
__global__ __launch_bounds__(kRouteWaves * kWave) void k_route_backward(RouteBwdArgs a)
{
    constexpr int TW = kWave / G, VE = Elem<DT>::kVE;
    constexpr uint32_t kNone = 0x7FFFDEADu;   // no choice: a NaN that no gradient has
    __shared__ uint32_t grads[kRouteWaves][TW * G * V];
    const int lane = lane_id(), wave = threadIdx.x / kWave, pos = lane % G, sub = lane / G;
    const int experts = a.experts, topk = a.topk;
    float load[V] = {}, zc = 0.0f;
    if (a.d_losses) {
        const int n = a.counts[experts];
        const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
        const float c = a.d_losses[0] * ((float)experts / (float)topk) * inv * inv;
        zc = 2.0f * a.d_losses[1] * inv;
#pragma unroll
        for (int i = 0; i < V; ++i)
            load[i] = pos * V + i < experts ? c * (float)a.counts[pos * V + i] : 0.0f;
    }
    uint32_t* grad = grads[wave];
    const size_t step = (size_t)gridDim.x * kRouteWaves * TW;
    for (size_t t0 = ((size_t)blockIdx.x * kRouteWaves + wave) * TW; t0 < a.tokens; t0 += step) {
        const size_t t = t0 + sub;
        const float lse = t < a.tokens ? a.lse[t] : -__builtin_inff();
        const bool live = lse != -__builtin_inff();
        float x[V];
        if (live)
            ld_logits<DT, V>(static_cast<const char*>(a.logits) + t * a.ld * Elem<DT>::kBytes, pos, experts, x);
        if (a.d_weights) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                grad[(sub * G + pos) * V + i] = kNone;
            wave_sync();
            const size_t left = a.tokens - t0;
            const int n = (left < (size_t)TW ? (int)left : TW) * topk;
            for (int i = lane; i < n; i += kWave) {
                const int id = a.ids[t0 * topk + i];
                if (id >= 0 && id < experts)
                    grad[i / topk * (G * V) + id] = __builtin_bit_cast(uint32_t, a.d_weights[t0 * topk + i]);
            }
            wave_sync();
        }
        float p[V], d[V], dot = 0.0f, share = 0.0f, mean = 0.0f;
        bool chosen[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = live && pos * V + i < experts ? expf(x[i] - lse) : 0.0f;
            const uint32_t g = a.d_weights ? grad[(sub * G + pos) * V + i] : kNone;
            chosen[i] = g != kNone;
            const float w = chosen[i] ? bits_f32(g) : 0.0f;
            d[i] = load[i];
            if (a.renormalize) {
                share += chosen[i] ? p[i] : 0.0f;
                mean += p[i] * w;
            } else {
                d[i] += w;
            }
            dot += p[i] * d[i];
            x[i] = w;
        }
        dot = group_sum<G>(dot);
        if (a.renormalize) {
            share = group_sum<G>(share);
            mean = group_sum<G>(mean);
            const float inv = share > 0.0f ? 1.0f / share : 0.0f;
            mean *= inv;
#pragma unroll
            for (int i = 0; i < V; ++i)
                d[i] += chosen[i] ? (x[i] - mean) * inv : 0.0f;
        }
        const float rest = (live ? zc * lse : 0.0f) - dot;
#pragma unroll
        for (int i = 0; i < V; ++i)
            d[i] = live ? p[i] * (d[i] + rest) : 0.0f;
        if (t < a.tokens)
#pragma unroll
            for (int i = 0; i < V / VE; ++i)
                st_row<DT, true>(static_cast<char*>(a.d_logits) + t * a.ld_d * Elem<DT>::kBytes, pos * (V / VE) + i, experts,
                                 pack<DT>(d + i * VE));
    }
}

// Lanes a token: eight logits each, sixteen beyond 512 experts.
int lanes_for(int experts)
{
    int g = 1;
    while (g < kWave && g * 8 < experts)
        g *= 2;
    return g;
}

// Workgroups of a call: every wave its tokens once, up to four workgroups a CU.
uint32_t route_grid(size_t tokens, int experts)
{
    const size_t per = (size_t)kRouteWaves * (kWave / lanes_for(experts));
    const size_t want = (tokens + per - 1) / per, most = 4 * (size_t)device_cu_count();
    return (uint32_t)(want < 1 ? 1 : want < most ? want : most);
}

template <int DT, bool SUMS>
const void* route_fn(int experts)
{
    if (experts > 512)
        return (const void*)k_route<DT, 64, 16, SUMS>;
    switch (lanes_for(experts)) {
    case 1: return (const void*)k_route<DT, 1, 8, SUMS>;
    case 2: return (const void*)k_route<DT, 2, 8, SUMS>;
    case 4: return (const void*)k_route<DT, 4, 8, SUMS>;
    case 8: return (const void*)k_route<DT, 8, 8, SUMS>;
    case 16: return (const void*)k_route<DT, 16, 8, SUMS>;
    case 32: return (const void*)k_route<DT, 32, 8, SUMS>;
    default: return (const void*)k_route<DT, 64, 8, SUMS>;
    }
}

template <int DT>
const void* route_backward_fn(int experts)
{
    if (experts > 512)
        return (const void*)k_route_backward<DT, 64, 16>;
    switch (lanes_for(experts)) {
    case 1: return (const void*)k_route_backward<DT, 1, 8>;
    case 2: return (const void*)k_route_backward<DT, 2, 8>;
    case 4: return (const void*)k_route_backward<DT, 4, 8>;
    case 8: return (const void*)k_route_backward<DT, 8, 8>;
    case 16: return (const void*)k_route_backward<DT, 16, 8>;
    case 32: return (const void*)k_route_backward<DT, 32, 8>;
    default: return (const void*)k_route_backward<DT, 64, 8>;
    }
}

}  // namespace

size_t route_workspace_words(size_t tokens, int experts)
{
    return 1 + (size_t)route_grid(tokens, experts) * (2 * (size_t)experts + 2);
}

hipError_t launch_route(const RouteArgs& in, int dtype, hipStream_t s)
{
    RouteArgs a = in;
    void* params[] = {&a};
    a.parts = route_grid(a.tokens, a.experts);
    const void* fn = a.counts ? dtype ? route_fn<1, true>(a.experts) : route_fn<0, true>(a.experts)
                     : dtype  ? route_fn<1, false>(a.experts)
                              : route_fn<0, false>(a.experts);
    const hipError_t e = launch_logged("k_route", fn, dim3(a.parts), dim3(kRouteWaves * kWave), params, s);
    if (e != hipSuccess || !a.counts)
        return e;
    return launch_logged("k_route_sums", (const void*)k_route_sums, dim3(1), dim3(1024), params, s);
}

hipError_t launch_route_backward(const RouteBwdArgs& in, int dtype, hipStream_t s)
{
    RouteBwdArgs a = in;
    void* params[] = {&a};
    const void* fn = dtype ? route_backward_fn<1>(a.experts) : route_backward_fn<0>(a.experts);
    return launch_logged("k_route_backward", fn, dim3(route_grid(a.tokens, a.experts)), dim3(kRouteWaves * kWave), params, s);
}

}  // namespace rx
