// api_layers.hip -- the C entry points of the router, the products with 4-bit
// weights and the layer norm (route.hip, gemm_fp4.hip, layer_norm.hip):
// validation, argument packing, launch. As in api.hip every check runs before
// the first launch.
#include <math.h>

#include "api_checks.hpp"

namespace {

using namespace rx;

constexpr size_t kMaxFp4K = (size_t)1 << 23;

bool route_sizes_ok(size_t tokens, int experts) { return tokens <= kMaxRows && experts >= 1 && experts <= kMaxExperts; }
bool topk_ok(int topk, int experts) { return topk >= 1 && topk <= kMaxTopk && topk <= experts; }
bool aligned8(const void* p) { return ((uintptr_t)p & 7u) == 0; }
bool group_ok(int g) { return g == 32 || g == 64 || g == 128; }

// Dropout's threshold 65536 p of a probability, and what a kept element is
// multiplied with; false where p is no probability below 1.
bool dropout_ok(float drop, uint32_t* threshold, float* gain)
{
    if (!(drop >= 0.0f) || !(drop < 1.0f))
        return false;
    const double t = nearbyint((double)drop * 65536.0);
    if (t > 65535.0)
        return false;
    *threshold = (uint32_t)t;
    *gain = (float)(65536.0 / (65536.0 - t));
    return true;
}

}  // namespace

extern "C" {

size_t rx_moe_route_workspace(size_t tokens, int experts)
{
    return route_sizes_ok(tokens, experts) ? route_workspace_words(tokens, experts) * sizeof(uint32_t) : 0;
}

rx_status_t rx_moe_route(const void* logits, size_t ld_logits, const unsigned char* token_mask, size_t tokens, int experts,
                         int topk, int renormalize, rx_dtype_t dtype, int* expert_ids, float* weights, float* lse,
                         int* counts, float* losses, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (tokens > 0 && (!logits || !expert_ids || !weights))
        return RX_ERR_NULL;
    if (!counts != !losses)
        return RX_ERR_NULL;
    if (!route_sizes_ok(tokens, experts) || !topk_ok(topk, experts) || bad_ld(ld_logits, (size_t)experts, tokens))
        return RX_ERR_ARG;
    if (!hp_type(dtype))
        return RX_ERR_DTYPE;
    if (!element_aligned(logits, dtype) || !aligned4(expert_ids) || !aligned4(weights) || !aligned4(lse) ||
        !aligned4(counts) || !aligned4(losses))
        return RX_ERR_ALIGN;
    if (counts) {
        if (!workspace)
            return RX_ERR_NULL;
        if (!aligned4(workspace))
            return RX_ERR_ALIGN;
        if (workspace_bytes < rx_moe_route_workspace(tokens, experts))
            return RX_ERR_ARG;
    }
    if (tokens == 0 && !counts)
        return RX_OK;
    RouteArgs a = {};
    a.logits = logits;
    a.mask = token_mask;
    a.ids = expert_ids;
    a.weights = weights;
    a.lse = lse;
    a.counts = counts;
    a.losses = losses;
    a.workspace = static_cast<uint32_t*>(workspace);
    a.ld = ld_logits;
    a.tokens = tokens;
    a.experts = experts;
    a.topk = topk;
    a.renormalize = renormalize != 0;
    return launched(launch_route(a, dt_index(dtype), stream));
}

rx_status_t rx_moe_route_backward(const void* logits, size_t ld_logits, const int* expert_ids, const float* lse,
                                  const int* counts, const float* d_weights, const float* d_losses, size_t tokens,
                                  int experts, int topk, int renormalize, rx_dtype_t dtype, void* d_logits,
                                  size_t ld_d_logits, hipStream_t stream)
{
    if (tokens > 0 && (!logits || !lse || !d_logits || (d_weights && !expert_ids) || (d_losses && !counts)))
        return RX_ERR_NULL;
    if (!route_sizes_ok(tokens, experts) || !topk_ok(topk, experts) || bad_ld(ld_logits, (size_t)experts, tokens) ||
        bad_ld(ld_d_logits, (size_t)experts, tokens))
        return RX_ERR_ARG;
    if (!hp_type(dtype))
        return RX_ERR_DTYPE;
    if (!element_aligned(logits, dtype) || !element_aligned(d_logits, dtype) || !aligned4(expert_ids) || !aligned4(lse) ||
        !aligned4(counts) || !aligned4(d_weights) || !aligned4(d_losses))
        return RX_ERR_ALIGN;
    if (tokens == 0)
        return RX_OK;
    RouteBwdArgs a = {};
    a.logits = logits;
    a.ids = expert_ids;
    a.lse = lse;
    a.counts = counts;
    a.d_weights = d_weights;
    a.d_losses = d_losses;
    a.d_logits = d_logits;
    a.ld = ld_logits;
    a.ld_d = ld_d_logits;
    a.tokens = tokens;
    a.experts = experts;
    a.topk = topk;
    a.renormalize = renormalize != 0;
    return launched(launch_route_backward(a, dt_index(dtype), stream));
}

rx_status_t rx_quant_fp4(const void* x, size_t ld_x, size_t rows, size_t k, rx_dtype_t dtype, int group, void* codes,
                         size_t ld_codes, float* scales, hipStream_t stream)
{
    if (rows > 0 && k > 0 && (!x || !codes || !scales))
        return RX_ERR_NULL;
    if (!group_ok(group) || rows > kMaxRows || k > kMaxFp4K || bad_ld(ld_x, k, rows) || bad_ld(ld_codes, (k + 1) / 2, rows))
        return RX_ERR_ARG;
    if (!hp_type(dtype))
        return RX_ERR_DTYPE;
    if (!element_aligned(x, dtype) || !aligned4(scales))
        return RX_ERR_ALIGN;
    if (rows == 0 || k == 0)
        return RX_OK;
    QuantFp4Args a = {};
    a.x = x;
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = scales;
    a.ld_x = ld_x;
    a.ld_codes = ld_codes;
    a.rows = rows;
    a.k = k;
    a.group = group;
    return launched(launch_quant_fp4(a, dt_index(dtype), stream));
}

rx_status_t rx_gemm_fp4(const void* a, size_t ld_a, const void* b, size_t ld_b, size_t stride_b, const float* b_scales,
                        int group, const int* offsets, int experts, size_t rows, size_t n, size_t k, rx_dtype_t dtype,
                        void* out, size_t ld_out, hipStream_t stream)
{
    if (rows > 0 && n > 0 && (!out || (k > 0 && (!a || !b || !b_scales))))
        return RX_ERR_NULL;
    if (!group_ok(group) || rows > kMaxRows || n >= ((size_t)1 << 31) || k > kMaxFp4K || experts < 1 ||
        experts > kMaxExperts || (!offsets && experts != 1) || (rows > 1 && ld_a >= kMaxGemmLd) ||
        (n > 1 && ld_b >= kMaxGemmLd) || bad_ld(ld_a, k, rows) || bad_ld(ld_b, (k + 31) / 32 * 16) ||
        bad_ld(ld_out, n, rows) || stride_b > kMaxLd * 16)
        return RX_ERR_ARG;
    if (!hp_type(dtype))
        return RX_ERR_DTYPE;
    if (!element_aligned(a, dtype) || !aligned16(b) || ld_b % 16 || stride_b % 16 || !aligned4(b_scales) ||
        !aligned4(offsets) || !element_aligned(out, dtype))
        return RX_ERR_ALIGN;
    // tiles of at least 16 x 128 outputs, 512 threads each: a launch's limit of 2^32 threads
    if ((rows / 16 + (size_t)experts + 1) * ((n + 127) / 128) >= ((size_t)1 << 23) - 16)
        return RX_ERR_ARG;
    if (rows == 0 || n == 0)
        return RX_OK;
    GemmFp4Args g = {};
    g.a = a;
    g.b = static_cast<const uint8_t*>(b);
    g.b_scales = b_scales;
    g.offsets = offsets;
    g.out = out;
    g.ld_a = rows > 1 ? ld_a : k;
    g.ld_b = n > 1 ? ld_b : (k + 31) / 32 * 16;
    g.stride_b = stride_b;
    g.ld_out = ld_out;
    g.rows = (uint32_t)rows;
    g.n = (uint32_t)n;
    g.k = (uint32_t)k;
    g.groups = (uint32_t)((k + group - 1) / group);
    g.experts = experts;
    g.group = group;
    return launched(launch_gemm_fp4(g, dt_index(dtype), stream));
}

rx_status_t rx_layer_norm(const void* const* srcs, int nsrc, size_t ld_src, const void* bias, const void* residual,
                          size_t ld_residual, const void* w, const void* b, float eps, float drop,
                          const unsigned long long* rng, size_t rows, size_t hidden, rx_dtype_t dtype, void* out_h,
                          size_t ld_h, void* out_z, size_t ld_z, float* mean, float* rstd, hipStream_t stream)
{
    const bool empty = rows == 0 || hidden == 0;   // no data: its pointers may be NULL
    uint32_t threshold = 0;
    float gain = 1.0f;
    if (!srcs || (!empty && !out_h && !out_z))
        return RX_ERR_NULL;
    if (nsrc < 1 || nsrc > RX_MAX_SRC || rows > kMaxRows || hidden > (size_t)kMaxNormHidden ||
        bad_ld(ld_src, hidden, rows) || (residual && bad_ld(ld_residual, hidden, rows)) ||
        (out_h && bad_ld(ld_h, hidden, rows)) || (out_z && bad_ld(ld_z, hidden, rows)) || !(eps > 0.0f) ||
        !isfinite(eps) || !dropout_ok(drop, &threshold, &gain))
        return RX_ERR_ARG;
    if (!hp_type(dtype))
        return RX_ERR_DTYPE;
    for (int j = 0; j < nsrc; ++j)
        if (!srcs[j] && !empty)
            return RX_ERR_NULL;
    if (threshold && !rng && !empty)
        return RX_ERR_NULL;
    for (int j = 0; j < nsrc; ++j)
        if (!element_aligned(srcs[j], dtype))
            return RX_ERR_ALIGN;
    const void* data[] = {bias, residual, w, b, out_h, out_z};
    for (const void* p : data)
        if (!element_aligned(p, dtype))
            return RX_ERR_ALIGN;
    if (!aligned4(mean) || !aligned4(rstd) || !aligned8(rng))
        return RX_ERR_ALIGN;
    if (empty)
        return RX_OK;
    LayerNormArgs a = {};
    for (int j = 0; j < nsrc; ++j)
        a.src[j] = srcs[j];
    a.bias = bias;
    a.residual = residual;
    a.w = w;
    a.b = b;
    a.rng = rng;
    a.out_h = out_h;
    a.out_z = out_z;
    a.mean = mean;
    a.rstd = rstd;
    a.ld_src = ld_src;
    a.ld_residual = ld_residual;
    a.ld_h = ld_h;
    a.ld_z = ld_z;
    a.rows = rows;
    a.hidden = hidden;
    a.threshold = threshold;
    a.gain = gain;
    a.eps = eps;
    a.inv_hidden = (float)(1.0 / (double)hidden);
    a.nsrc = nsrc;
    return launched(launch_layer_norm(a, dt_index(dtype), stream));
}

size_t rx_layer_norm_backward_workspace(size_t rows, size_t hidden)
{
    if (rows > kMaxRows || hidden > (size_t)kMaxNormHidden)
        return 0;
    return layer_norm_backward_floats(rows, hidden) * sizeof(float);
}

rx_status_t rx_layer_norm_backward(const void* h, size_t ld_h, const void* w, const float* mean, const float* rstd,
                                   float drop, const unsigned long long* rng, size_t rows, size_t hidden,
                                   rx_dtype_t dtype, const void* d_h, size_t ld_d_h, const void* d_z, size_t ld_d_z,
                                   void* d_src, size_t ld_d_src, void* d_residual, size_t ld_d_residual, float* d_bias,
                                   float* d_w, float* d_b, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    const bool empty = rows == 0 || hidden == 0;
    uint32_t threshold = 0;
    float gain = 1.0f;
    if (!empty && d_z && (!h || !mean || !rstd))
        return RX_ERR_NULL;
    if (rows > kMaxRows || hidden > (size_t)kMaxNormHidden || (h && bad_ld(ld_h, hidden, rows)) ||
        (d_h && bad_ld(ld_d_h, hidden, rows)) || (d_z && bad_ld(ld_d_z, hidden, rows)) ||
        (d_src && bad_ld(ld_d_src, hidden, rows)) || (d_residual && bad_ld(ld_d_residual, hidden, rows)) ||
        (!empty && d_src && d_src == d_residual) || !dropout_ok(drop, &threshold, &gain))
        return RX_ERR_ARG;
    if (!hp_type(dtype))
        return RX_ERR_DTYPE;
    if (threshold && !rng && !empty)
        return RX_ERR_NULL;
    const void* data[] = {h, w, d_h, d_z, d_src, d_residual};
    for (const void* p : data)
        if (!element_aligned(p, dtype))
            return RX_ERR_ALIGN;
    const void* f32[] = {mean, rstd, d_bias, d_w, d_b};
    for (const void* p : f32)
        if (!aligned4(p))
            return RX_ERR_ALIGN;
    if (!aligned8(rng))
        return RX_ERR_ALIGN;
    const size_t need = rx_layer_norm_backward_workspace(rows, hidden);
    if (need) {
        if (!workspace)
            return RX_ERR_NULL;
        if (!aligned16(workspace))
            return RX_ERR_ALIGN;
        if (workspace_bytes < need)
            return RX_ERR_ARG;
    }
    if (hidden == 0 || (rows == 0 && !d_bias && !d_w && !d_b))
        return RX_OK;
    LayerNormBwdArgs a = {};
    a.h = h;
    a.w = w;
    a.mean = mean;
    a.rstd = rstd;
    a.rng = rng;
    a.d_h = d_h;
    a.d_z = d_z;
    a.d_src = d_src;
    a.d_residual = d_residual;
    a.d_bias = d_bias;
    a.d_w = d_w;
    a.d_b = d_b;
    a.means = static_cast<float*>(workspace);
    a.ld_h = ld_h;
    a.ld_d_h = ld_d_h;
    a.ld_d_z = ld_d_z;
    a.ld_d_src = ld_d_src;
    a.ld_d_residual = ld_d_residual;
    a.rows = rows;
    a.hidden = hidden;
    a.threshold = threshold;
    a.gain = gain;
    a.inv_hidden = (float)(1.0 / (double)hidden);
    return launched(launch_layer_norm_backward(a, dt_index(dtype), stream));
}

}  // extern "C"
