// route.hip -- each token's experts from the router's logits, the counts and
// the losses over all tokens, and their gradient (gfx950). Defined in rx.h.
//
// G lanes hold a token's logits, V neighbouring ones each, and a wave 64 / G
// tokens: a maximum over a token costs log2 G steps between lanes and V / 2
// within one, so few lanes with many logits each are cheaper than a wave a
// token. A lane keeps the same experts for all its tokens, so the sums over
// the tokens stay in its registers and meet in LDS at the end. 16384 x 128 BF16,
// top 8, takes 9.8 us forward, the sums 4.2 and the gradient 5.9, where the bytes would
// take 1.6: 185 vector instructions a token are about half of the forward's, the
// rest is the wait of one choice for the one before, with two waves a SIMD (waves wait 44% of their cycles).
#include "block_common.hpp"

namespace rx {
namespace {

// Logits pos V .. pos V + V - 1 of a row: the loads, which wait for nothing, and
// their values.
template <int DT, int V> struct RawLogits { u32x4 v[V / Elem<DT>::kVE]; };

template <int DT, int G, int V>   // more than one lane: more than a vector of experts
__device__ __forceinline__ RawLogits<DT, V> ld_logits(const void* row, int pos, int experts)
{
    constexpr int N = V / Elem<DT>::kVE;
    RawLogits<DT, V> r;
#pragma unroll
    for (int i = 0; i < N; ++i)
        r.v[i] = ld_raw<DT, true, false, G == 1>(row, pos * N + i, experts);
    return r;
}
template <int DT, int V>
__device__ __forceinline__ void logits_of(const RawLogits<DT, V>& r, int pos, int experts, float* x)
{
    constexpr int VE = Elem<DT>::kVE, N = V / VE;
#pragma unroll
    for (int i = 0; i < N; ++i)
        unpack<DT>(fixed<DT, true>(r.v[i], pos * N + i, experts), x + i * VE);
}

// Unsigned numbers in the logits' order, the lower expert's above its equal's: what
// is taken or past the experts is 0, -inf at most kKeyNone, NaN above all; -0
// equals 0. A BF16 logit leaves 16 bits for its expert, so that one comparison
// finds the largest and its place.
constexpr uint32_t kKeyNone = 0x007FFFFFu;
template <int DT>
__device__ __forceinline__ uint32_t key_of(float x, int expert)
{
    uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
    u = x != x ? 0x7FC00000u : u;
    u ^= (uint32_t)((int32_t)u >> 31) | 0x80000000u;
    return DT == 0 ? u : (u & 0xFFFF0000u) | (0xFFFFu - (uint32_t)expert);
}
template <int DT>
__device__ __forceinline__ float value_of(uint32_t key)
{
    const uint32_t u = key ^ (key >> 31 ? 0x80000000u : 0xFFFFFFFFu);
    return bits_f32(DT == 0 ? u : u & 0xFFFF0000u);
}

// exp of d <= 0 in six instructions: 2^y with y the rounded d log2 e, and what the
// rounding left as a factor of 1 + r ln 2. v_exp_f32 is within a unit, the factor
// within half of one; values below 2^-126 become 0, and a NaN too. For the sums over a
// token: a weight's own numerator takes expf.
__device__ __forceinline__ float exp_of(float d)
{
    d = fmaxf(d, -150.0f);
    const float y = d * 1.44269502f;
    const float r = __builtin_fmaf(d, 1.92596299e-8f, __builtin_fmaf(d, 1.44269502f, -y));
    const float e = __builtin_amdgcn_exp2f(y);
    return __builtin_fmaf(e, r * 0.693147182f, e);
}

// The workspace: a counter; for each workgroup a part (experts counts, experts
// sums of P), then for each its tokens and the sum of their lse^2; and a sum for
// each workgroup of the second launch.
__device__ __host__ __forceinline__ size_t part_words(int experts) { return 2 * (size_t)experts; }
constexpr int kSumExperts = 32;   // of a workgroup of the second launch

// The losses from n tokens, the sum over the experts of count times sum of P,
// and the sum of lse^2.
__device__ __forceinline__ void put_losses(const RouteArgs& a, uint32_t n, float dot, float z)
{
    const float inv = n ? 1.0f / (float)n : 0.0f;
    a.counts[a.experts] = (int)n;
    a.losses[0] = dot * inv * inv * ((float)a.experts / (float)a.topk);
    a.losses[1] = z * inv;
}

// A workgroup's waves at most: with sums what the registers allow, without four.
template <int V, bool SUMS> constexpr int kRouteWaves = !SUMS ? 4 : V == 16 ? 8 : 16;

template <int DT, int G, int V, bool SUMS>
__global__ __launch_bounds__((kRouteWaves<V, SUMS> * kWave)) void k_route(RouteArgs a)
{
    constexpr int TW = kWave / G;                                // tokens of a wave
    constexpr int MOST = V * G < kMaxTopk ? V * G : kMaxTopk;    // choices of a token
    constexpr int W = kRouteWaves<V, SUMS>;
    struct Pick {
        int id;
        uint32_t key;
    };
    __shared__ Pick picks[W][TW * MOST];
    // without sums a CU has room for as many workgroups as the registers leave (eight, or four)
    static_assert(SUMS || sizeof(picks) * (V == 16 ? 4 : 8) <= 160 * 1024, "");
    __shared__ uint32_t sums[SUMS ? 2 : 1][SUMS ? W : 1][SUMS ? V * G : 1];
    __shared__ uint32_t totals[W][2];
    __shared__ float dots[W];
    const int lane = lane_id(), wave = threadIdx.x / kWave, waves = blockDim.x / kWave, pos = lane % G, sub = lane / G;
    const int experts = a.experts, topk = a.topk;
    float prob[V] = {}, squares = 0.0f;
    uint32_t count[V] = {}, live_tokens = 0;
    const size_t step = (size_t)gridDim.x * waves * TW;
    for (size_t t0 = ((size_t)blockIdx.x * waves + wave) * TW; t0 < a.tokens; t0 += step) {
        const size_t t = t0 + sub;
        // an empty token's logits are loaded too: no wait for the mask
        const RawLogits<DT, V> raw =
            ld_logits<DT, G, V>(static_cast<const char*>(a.logits) + (t < a.tokens ? t : a.tokens - 1) * a.ld * Elem<DT>::kBytes, pos, experts);
        bool live = t < a.tokens && (!a.mask || a.mask[t]);
        float x[V];
        uint32_t key[V];
        logits_of<DT, V>(raw, pos, experts, x);
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            key[i] = live && pos * V + i < experts ? key_of<DT>(x[i], pos * V + i) : 0;
            mine = umax(mine, key[i]);
        }
        uint32_t top = group_max<G>(mine);
        live = top > kKeyNone;
        const float high = live ? value_of<DT>(top) : 0.0f;
        float sum = 0.0f, e[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            e[i] = exp_of(key[i] ? x[i] - high : -__builtin_inff());   // 0 for an empty token
            sum += e[i];
        }
        sum = group_sum<G>(sum);
        // the choices, one a round; what is taken has no key any more
        Pick* pick = picks[wave] + sub * topk;
        uint32_t kept = 0;   // logits that can be taken
#pragma unroll
        for (int i = 0; i < V; ++i)
            kept |= key[i] > kKeyNone ? 1u << i : 0;
        for (int j = 0; j < topk; ++j) {
            if constexpr (DT == 0) {
                const uint64_t owners = __ballot(mine == top) >> (sub * G);
                bool mayhave = pos == __builtin_ctzll(owners);
                int id = -1;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const bool hit = mayhave && key[i] == top;   // the first of equals
                    mayhave = mayhave && !hit;
                    id = hit ? i : id;
                    key[i] = hit ? 0 : key[i];
                }
                if (id >= 0)
                    pick[j] = Pick{pos * V + id, top};
            } else {
                if (pos == 0)
                    pick[j] = Pick{(int)(0xFFFFu - (top & 0xFFFFu)), top};
#pragma unroll
                for (int i = 0; i < V; ++i)
                    key[i] = key[i] == top ? 0 : key[i];
            }
            mine = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                mine = umax(mine, key[i]);
            top = group_max<G>(mine);
        }
        uint32_t taken = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            taken |= key[i] == 0 ? kept & 1u << i : 0;
        float chosen = sum;
        if (a.renormalize) {
            chosen = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                chosen += taken >> i & 1 ? e[i] : 0.0f;
            chosen = group_sum<G>(chosen);
        }
        const float scale = live ? chosen : 1.0f;
        const float lse = live ? high + logf(sum) : -__builtin_inff();
        if (a.lse && pos == 0 && t < a.tokens)
            a.lse[t] = lse;
        // tokens of the wave follow each other: their choices too
        const size_t left = a.tokens - t0;
        const int n = (left < (size_t)TW ? (int)left : TW) * topk;
        wave_sync();
        for (int i0 = 0; i0 < n; i0 += kWave) {
            const int i = i0 + lane;
            // the largest logit and the divisor of the token that choice i belongs to
            const int from = (i < n ? i / topk : 0) * G * 4;
            const float top_of = bits_f32((uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)__builtin_bit_cast(uint32_t, high)));
            const float div = bits_f32((uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)__builtin_bit_cast(uint32_t, scale)));
            if (i < n) {
                const Pick p = picks[wave][i];
                const bool some = p.key > kKeyNone;
                a.ids[t0 * topk + i] = some ? p.id : -1;
                a.weights[t0 * topk + i] = some ? expf(value_of<DT>(p.key) - top_of) / div : 0.0f;
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
                squares += lse * lse;
                ++live_tokens;
            }
        }
    }
    if constexpr (SUMS) {
        // over the wave's groups, then over the waves, in their order
        const bool alone = gridDim.x == 1;
        uint32_t* out = a.workspace + 1 + blockIdx.x * part_words(experts);
        if (blockIdx.x == 0 && threadIdx.x == 0)
            a.workspace[0] = 0;   // the second launch's counter
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c = across<G>(count[i]), p = __builtin_bit_cast(uint32_t, across<G>(prob[i]));
            if (sub == 0) {
                sums[0][wave][pos * V + i] = c;
                sums[1][wave][pos * V + i] = p;
            }
        }
        squares = wave_sum(squares);
        live_tokens = wave_sum_u(live_tokens);
        if (lane == 0) {
            totals[wave][0] = live_tokens;
            totals[wave][1] = __builtin_bit_cast(uint32_t, squares);
        }
        __syncthreads();
        float dot = 0.0f;
        for (int e = threadIdx.x; e < experts; e += blockDim.x) {
            uint32_t c = 0;
            float p = 0.0f;
            for (int w = 0; w < waves; ++w) {
                c += sums[0][w][e];
                p += bits_f32(sums[1][w][e]);
            }
            dot += (float)c * p;
            if (alone) {
                a.counts[e] = (int)c;
            } else {
                out[e] = c;
                out[experts + e] = __builtin_bit_cast(uint32_t, p);
            }
        }
        if (alone) {
            dot = wave_sum(dot);
            if (lane == 0)
                dots[wave] = dot;
            __syncthreads();
        }
        if (threadIdx.x == 0) {
            uint32_t n = 0;
            float z = 0.0f, d = 0.0f;
            for (int w = 0; w < waves; ++w) {
                n += totals[w][0];
                z += bits_f32(totals[w][1]);
                d += alone ? dots[w] : 0.0f;
            }
            if (alone) {
                put_losses(a, n, d, z);
            } else {
                out = a.workspace + 1 + a.parts * part_words(experts) + 2 * blockIdx.x;
                out[0] = n;
                out[1] = __builtin_bit_cast(uint32_t, z);
            }
        }
    }
}

// The workgroups' parts in their order: 32 experts a workgroup, half the lanes for
// the counts and half for the sums of P, the parts dealt to 16 waves, 16 of a
// wave's loads at a time. The last workgroup to come adds the workgroups' share of
// the loss.
__global__ __launch_bounds__(1024) void k_route_sums(RouteArgs a)
{
    __shared__ uint32_t sums[16][kWave], n_of[16], order;
    __shared__ float z_of[16];
    const int experts = a.experts, lane = lane_id(), wave = threadIdx.x / kWave;
    const int e = (int)blockIdx.x * kSumExperts + lane % kSumExperts;
    const bool counts = lane < kSumExperts;
    const size_t words = part_words(experts);
    const uint32_t *in = a.workspace + 1, *totals = in + a.parts * words;
    float* shares = reinterpret_cast<float*>(a.workspace + 1 + a.parts * (words + 2));
    const uint32_t* at = in + (counts ? 0 : experts) + (e < experts ? e : 0);
    uint32_t n = 0, c = 0;
    float z = 0.0f, p = 0.0f;
    if (threadIdx.x < a.parts) {   // at most 1024
        n = totals[2 * threadIdx.x];
        z = bits_f32(totals[2 * threadIdx.x + 1]);
    }
    for (uint32_t g0 = wave; g0 < a.parts; g0 += 256) {
        uint32_t x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t g = g0 + 16 * i;
            x[i] = at[(g < a.parts ? g : g0) * words];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (g0 + 16 * i < a.parts) {
                c += x[i];
                p += bits_f32(x[i]);
            }
    }
    sums[wave][lane] = counts ? c : __builtin_bit_cast(uint32_t, p);
    n = wave_sum_u(n);
    z = wave_sum(z);
    if (lane == 0) {
        n_of[wave] = n;
        z_of[wave] = z;
    }
    __syncthreads();
    if (wave)
        return;
    c = n = 0;
    p = z = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        c += sums[w][lane % kSumExperts];
        p += bits_f32(sums[w][kSumExperts + lane % kSumExperts]);
        n += n_of[w];
        z += z_of[w];
    }
    if (counts && e < experts)
        a.counts[e] = (int)c;
    float dot = wave_sum(counts && e < experts ? (float)c * p : 0.0f);
    if (gridDim.x > 1) {
        if (lane == 0) {
            __hip_atomic_store(&shares[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            order = __hip_atomic_fetch_add(&a.workspace[0], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
        }
        wave_sync();
        if (order != gridDim.x - 1)
            return;
        // at most 32 shares, a lane each
        dot = wave_sum((uint32_t)lane < gridDim.x ? __hip_atomic_load(&shares[lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0f);
    }
    if (lane == 0)
        put_losses(a, n, dot, z);
}

// ---- gradient ------------------------------------------------------------------

// dl = P (c f + h - A + z), with c f from the counts, h and A from the weights'
// gradients: an element of the token's choices in LDS at a time.
template <int DT, int G, int V>
__global__ __launch_bounds__(256) void k_route_backward(RouteBwdArgs a)
{
    constexpr int TW = kWave / G, VE = Elem<DT>::kVE, kWaves = 4;
    constexpr uint32_t kNone = 0x7FFFDEADu;   // no choice; a gradient that is NaN is kNaN
    constexpr uint32_t kNaN = 0x7FC00000u;
    __shared__ __align__(16) uint32_t grads[kWaves][TW * G * V];
    const int lane = lane_id(), wave = threadIdx.x / kWave, pos = lane % G, sub = lane / G;
    const int experts = a.experts, topk = a.topk;
    float load[V] = {}, zc = 0.0f;
    uint32_t* grad = grads[wave];
    const size_t step = (size_t)gridDim.x * kWaves * TW;
    bool first = true;
    for (size_t t0 = ((size_t)blockIdx.x * kWaves + wave) * TW; t0 < a.tokens; t0 += step) {
        // all loads before anything waits
        const size_t t = t0 + sub, row = t < a.tokens ? t : a.tokens - 1;
        const RawLogits<DT, V> raw = ld_logits<DT, G, V>(static_cast<const char*>(a.logits) + row * a.ld * Elem<DT>::kBytes, pos, experts);
        const float stored = a.lse[row], lse = t < a.tokens ? stored : -__builtin_inff();
        const size_t left = a.tokens - t0;
        const int n = (left < (size_t)TW ? (int)left : TW) * topk;
        int id = -1;
        float dw = 0.0f;
        if (a.d_weights) {
            const size_t at = t0 * topk + (lane < n ? lane : 0);
            id = a.ids[at];
            dw = a.d_weights[at];
        }
        if (first && a.d_losses) {
            u32x4 c[V / 4];
#pragma unroll
            for (int i = 0; i < V / 4; ++i)
                c[i] = ld_raw<0, true, false, G == 1>(a.counts, pos * (V / 4) + i, experts);
            const int tokens = a.counts[experts];
            const float d0 = a.d_losses[0], d1 = a.d_losses[1], inv = tokens > 0 ? 1.0f / (float)tokens : 0.0f;
            const float by = d0 * ((float)experts / (float)topk) * inv * inv;
            zc = 2.0f * d1 * inv;
#pragma unroll
            for (int i = 0; i < V; ++i)   // 0 past the experts
                load[i] = by * (float)(int)fixed<0, true>(c[i / 4], pos * (V / 4) + i / 4, experts)[i % 4];
        }
        first = false;
        const bool live = lse != -__builtin_inff();
        float x[V];
        logits_of<DT, V>(raw, pos, experts, x);
        if (a.d_weights) {
            wave_sync();
#pragma unroll
            for (int i = 0; i < V; ++i)
                grad[(sub * G + pos) * V + i] = kNone;
            wave_sync();
            for (int i = lane; i < n; i += kWave) {
                if (i >= kWave) {
                    id = a.ids[t0 * topk + i];
                    dw = a.d_weights[t0 * topk + i];
                }
                if (i < n && id >= 0 && id < experts)
                    grad[i / topk * (G * V) + id] = dw != dw ? kNaN : __builtin_bit_cast(uint32_t, dw);
            }
            wave_sync();
        }
        u32x4 got[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            got[i] = u32x4{kNone, kNone, kNone, kNone};
        if (a.d_weights)
#pragma unroll
            for (int i = 0; i < V / 4; ++i)
                got[i] = *reinterpret_cast<const u32x4*>(&grad[(sub * G + pos) * V + 4 * i]);
        float p[V], d[V], dot = 0.0f, share = 0.0f, mean = 0.0f;
        bool chosen[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = expf(live && pos * V + i < experts ? x[i] - lse : -__builtin_inff());
            const uint32_t g = got[i / 4][i % 4];
            chosen[i] = g != kNone;
            const float w = chosen[i] ? bits_f32(g) : 0.0f;
            share += chosen[i] ? p[i] : 0.0f;
            mean += p[i] * w;
            d[i] = load[i] + (a.renormalize ? 0.0f : w);
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

// Lanes a token with v logits each.
int lanes_for(int experts, int v)
{
    int g = 1;
    while (g < kWave && g * v < experts)
        g *= 2;
    return g;
}

// Waves and workgroups of a call, and the logits of a lane. Sixteen logits a lane
// cost a token less (a round of choices 46 instructions for twice the tokens
// instead of 38), eight have more waves and a shorter way: sixteen beyond 512
// experts, and where eight would take over twelve waves a CU (16384 x
// 128 BF16 with sums: 10.3 against 11.2 us).
// With sums a workgroup a CU, so that there are few parts to add, and one for up
// to 16 waves of tokens, which then needs no second launch; without, four waves a
// workgroup.
struct Spread {
    int v;
    unsigned threads;
    uint32_t grid;
};
Spread spread(size_t tokens, int experts, bool sums)
{
    const size_t all = (size_t)device_cu_count(), cus = !sums ? 8 * all : all < 1024 ? all : 1024;
    auto units_of = [&](int v) {
        const size_t per = (size_t)(kWave / lanes_for(experts, v));
        return tokens ? (tokens + per - 1) / per : 1;
    };
    const int v = experts > 512 || units_of(8) > 12 * all ? 16 : 8;
    const size_t units = units_of(v), most = !sums ? kRouteWaves<8, false> : v == 16 ? kRouteWaves<16, true> : kRouteWaves<8, true>;
    size_t w = units < most ? units : most;
    if (sums && units > most) {   // every CU before a second wave on one
        w = (units + cus - 1) / cus;
        w = w < 4 ? 4 : w < most ? w : most;
    }
    const size_t want = (units + w - 1) / w;
    return {v, (unsigned)(w * kWave), (uint32_t)(want < cus ? want : cus)};
}

template <int DT, bool SUMS, int V>
const void* route_fn(int experts)
{
    switch (lanes_for(experts, V)) {
    case 1: return (const void*)k_route<DT, 1, V, SUMS>;
    case 2: return (const void*)k_route<DT, 2, V, SUMS>;
    case 4: return (const void*)k_route<DT, 4, V, SUMS>;
    case 8: return (const void*)k_route<DT, 8, V, SUMS>;
    case 16: return (const void*)k_route<DT, 16, V, SUMS>;
    case 32: return (const void*)k_route<DT, 32, V, SUMS>;
    default: return (const void*)k_route<DT, 64, V, SUMS>;
    }
}
template <int DT>
const void* route_fn(int experts, int v, bool sums)
{
    return v == 16 ? sums ? route_fn<DT, true, 16>(experts) : route_fn<DT, false, 16>(experts)
                   : sums ? route_fn<DT, true, 8>(experts) : route_fn<DT, false, 8>(experts);
}

template <int DT>
const void* route_backward_fn(int experts)
{
    if (experts > 512)
        return (const void*)k_route_backward<DT, 64, 16>;
    switch (lanes_for(experts, 8)) {
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
    return 1 + spread(tokens, experts, true).grid * (part_words(experts) + 2) + (size_t)(experts + kSumExperts - 1) / kSumExperts;
}

hipError_t launch_route(const RouteArgs& in, int dtype, hipStream_t s)
{
    RouteArgs a = in;
    void* params[] = {&a};
    const Spread sp = spread(a.tokens, a.experts, a.counts);
    a.parts = sp.grid;
    const void* fn = dtype ? route_fn<1>(a.experts, sp.v, a.counts) : route_fn<0>(a.experts, sp.v, a.counts);
    const hipError_t e = launch_logged("k_route", fn, dim3(sp.grid), dim3(sp.threads), params, s);
    if (e != hipSuccess || !a.counts || sp.grid == 1)
        return e;
    return launch_logged("k_route_sums", (const void*)k_route_sums, dim3((unsigned)(a.experts + kSumExperts - 1) / kSumExperts), dim3(1024), params, s);
}

hipError_t launch_route_backward(const RouteBwdArgs& in, int dtype, hipStream_t s)
{
    RouteBwdArgs a = in;
    void* params[] = {&a};
    const void* fn = dtype ? route_backward_fn<1>(a.experts) : route_backward_fn<0>(a.experts);
    const size_t per = 4 * (size_t)(kWave / lanes_for(a.experts, a.experts > 512 ? 16 : 8));   // tokens of a workgroup
    const size_t want = (a.tokens + per - 1) / per, most = 8 * (size_t)device_cu_count();
    return launch_logged("k_route_backward", fn, dim3((unsigned)(want < most ? want : most)), dim3(256), params, s);
}

}  // namespace rx
