// api_block.hip -- the C entry points of the operators around a block's
// allreduce (moe.hip, norm.hip, gemm_i8.hip): validation, argument packing,
// launch. As in api.hip every check runs before the first launch.
#include <math.h>

#include "api_checks.hpp"

namespace {

using namespace rx;

bool dispatch_sizes_ok(size_t tokens, int topk, int experts)
{
    return topk >= 1 && topk <= kMaxTopk && experts >= 1 && experts <= kMaxExperts && tokens <= kMaxRows &&
           tokens * (size_t)topk < ((size_t)1 << 31);
}

size_t gate_rows_or_one(size_t gate_rows, size_t rows)
{
    return gate_rows < 1 ? 1 : gate_rows < rows ? gate_rows : rows < 1 ? 1 : rows;
}

}  // namespace

extern "C" {

// Above kDispatchCountAll pairs a caller always brings one, also up to the
// number that the placing kernel still counts by itself (moe.hip), so that this
// limit can move without a caller's noticing.
size_t rx_moe_dispatch_workspace(size_t tokens, int topk, int experts)
{
    if (!dispatch_sizes_ok(tokens, topk, experts) || tokens * (size_t)topk <= kDispatchCountAll)
        return 0;
    const size_t pairs = tokens * (size_t)topk, seg = dispatch_segment(pairs);
    return (size_t)experts * ((pairs + seg - 1) / seg + 1) * sizeof(uint32_t);   // a row to spare
}

rx_status_t rx_moe_dispatch(const int* expert_ids, size_t tokens, int topk, int first_expert, int experts,
                            const void* x, size_t ld_x, size_t hidden, rx_dtype_t x_dtype, int* offsets, int* order,
                            int* slots, void* rows, size_t ld_rows, rx_dtype_t rows_dtype, float* row_scales,
                            void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!offsets || (tokens > 0 && (!expert_ids || !order || !slots)))
        return RX_ERR_NULL;
    if (!dispatch_sizes_ok(tokens, topk, experts) || first_expert < 0 || first_expert > INT32_MAX - experts)
        return RX_ERR_ARG;
    const bool gather = x || rows || row_scales;
    const bool quant = gather && rows_dtype == RX_INT8;
    if (gather) {
        if (!x || !rows || (quant && !row_scales))
            return RX_ERR_NULL;
        if (!quant && row_scales)
            return RX_ERR_ARG;
        if (hidden > kMaxHidden || bad_ld(ld_x, hidden, tokens) || bad_ld(ld_rows, hidden, tokens * (size_t)topk))
            return RX_ERR_ARG;
        if (!hp_type(x_dtype) || (!quant && rows_dtype != x_dtype))
            return RX_ERR_DTYPE;
        if (!element_aligned(x, x_dtype) || !element_aligned(rows, rows_dtype) || (quant && !aligned4(row_scales)))
            return RX_ERR_ALIGN;
    }
    if (!aligned4(offsets) || !aligned4(expert_ids) || !aligned4(order) || !aligned4(slots))
        return RX_ERR_ALIGN;
    const size_t need = rx_moe_dispatch_workspace(tokens, topk, experts);
    if (need) {
        if (!workspace)
            return RX_ERR_NULL;
        if (!aligned4(workspace))
            return RX_ERR_ALIGN;
        if (workspace_bytes < need)
            return RX_ERR_ARG;
    }
    DispatchArgs a = {};
    a.ids = expert_ids;
    a.offsets = offsets;
    a.order = order;
    a.slots = slots;
    a.x = x;
    a.rows = rows;
    a.row_scales = row_scales;
    a.ld_x = ld_x;
    a.ld_rows = ld_rows;
    a.hidden = hidden;
    a.tokens = (uint32_t)tokens;
    a.pairs = (uint32_t)(tokens * (size_t)topk);
    a.segment = dispatch_segment(a.pairs);
    a.segments = (a.pairs + a.segment - 1) / a.segment;
    a.counts = static_cast<uint32_t*>(workspace);
    a.topk = topk;
    a.first = first_expert;
    a.experts = experts;
    return launched(launch_dispatch(a, gather ? dt_index(x_dtype) : 0, !gather ? 0 : quant ? 2 : 1, stream));
}

rx_status_t rx_moe_combine(const void* rows, size_t ld_rows, size_t nrows, const int* slots, const float* weights,
                           size_t tokens, int topk, size_t hidden, rx_dtype_t dtype, void* out, size_t ld_out,
                           hipStream_t stream)
{
    if (tokens > 0 && hidden > 0 && (!slots || !out || (nrows > 0 && !rows)))
        return RX_ERR_NULL;
    if (topk < 1 || topk > kMaxTopk || tokens > kMaxRows || nrows >= ((size_t)1 << 31) || hidden > kMaxHidden ||
        bad_ld(ld_rows, hidden, nrows) || bad_ld(ld_out, hidden, tokens) ||
        tokens * ((hidden + 255) / 256) >= ((size_t)1 << 26))   // a wave for every 64 vectors
        return RX_ERR_ARG;
    if (!hp_type(dtype))
        return RX_ERR_DTYPE;
    if (!element_aligned(rows, dtype) || !element_aligned(out, dtype) || !aligned4(slots) || !aligned4(weights))
        return RX_ERR_ALIGN;
    if (tokens == 0 || hidden == 0)
        return RX_OK;
    CombineArgs a = {};
    a.rows = rows;
    a.slots = slots;
    a.weights = weights;
    a.out = out;
    a.ld_rows = ld_rows;
    a.ld_out = ld_out;
    a.nrows = nrows;
    a.tokens = tokens;
    a.hidden = hidden;
    a.topk = topk;
    return launched(launch_combine(a, dt_index(dtype), stream));
}

rx_status_t rx_moe_combine_backward(const void* d_out, size_t ld_d_out, const void* rows, size_t ld_rows,
                                    size_t nrows, const int* slots, const float* weights, const int* kept,
                                    size_t tokens, int topk, size_t hidden, rx_dtype_t dtype, void* d_rows,
                                    size_t ld_d_rows, float* d_weights, hipStream_t stream)
{
    const bool clears = nrows > 0 && hidden > 0;   // rows that no pair owns, also without tokens
    if ((tokens > 0 && (!slots || !kept)) || (clears && (!kept || !d_rows)))
        return RX_ERR_NULL;
    if (tokens > 0 && hidden > 0 && (!d_out || (nrows > 0 && d_weights && !rows)))
        return RX_ERR_NULL;
    if (topk < 1 || topk > kMaxTopk || tokens > kMaxRows || nrows >= ((size_t)1 << 31) || hidden > kMaxHidden ||
        bad_ld(ld_d_out, hidden, tokens) || bad_ld(ld_d_rows, hidden, nrows) ||
        (d_weights && bad_ld(ld_rows, hidden, nrows)))
        return RX_ERR_ARG;
    if (!hp_type(dtype))
        return RX_ERR_DTYPE;
    if (!element_aligned(d_out, dtype) || !element_aligned(rows, dtype) || !element_aligned(d_rows, dtype) ||
        !aligned4(slots) || !aligned4(weights) || !aligned4(kept) || !aligned4(d_weights))
        return RX_ERR_ALIGN;
    // without a device there is no memory that the rows could lie in: a call without tokens succeeds there
    int device;
    if (tokens == 0 && (!clears || hipGetDevice(&device) != hipSuccess))
        return RX_OK;
    CombineBwdArgs a = {};
    a.d_out = d_out;
    a.rows = rows;
    a.slots = slots;
    a.weights = weights;
    a.kept = kept;
    a.d_rows = d_rows;
    a.d_weights = d_weights;
    a.ld_d_out = ld_d_out;
    a.ld_rows = ld_rows;
    a.ld_d_rows = ld_d_rows;
    a.nrows = nrows;
    a.tokens = tokens;
    a.hidden = hidden;
    a.topk = topk;
    return launched(launch_combine_backward(a, dt_index(dtype), stream));
}

rx_status_t rx_residual_norm(const void* const* srcs, int nsrc, size_t ld_src, const void* residual,
                             size_t ld_residual, const void* gate, size_t gate_rows, const void* w_post,
                             const void* w_pre, float residual_scale, float eps, size_t rows, size_t hidden,
                             rx_dtype_t dtype, void* out_h, size_t ld_h, void* out_z, size_t ld_z, float* rstd_post,
                             float* rstd_pre, hipStream_t stream)
{
    const bool empty = rows == 0 || hidden == 0;   // no data: its pointers may be NULL
    if (!srcs || (!empty && !out_h && !out_z) || (!empty && out_z && !w_pre))
        return RX_ERR_NULL;
    if (nsrc < 1 || nsrc > RX_MAX_SRC || rows > kMaxRows || hidden > (size_t)kMaxNormHidden ||
        bad_ld(ld_src, hidden, rows) || (residual && bad_ld(ld_residual, hidden, rows)) ||
        (out_h && bad_ld(ld_h, hidden, rows)) || (out_z && bad_ld(ld_z, hidden, rows)) || (gate && gate_rows < 1) ||
        !(eps > 0.0f) || !isfinite(eps) || !isfinite(residual_scale))
        return RX_ERR_ARG;
    if (!hp_type(dtype))
        return RX_ERR_DTYPE;
    for (int j = 0; j < nsrc; ++j)
        if (!srcs[j] && !empty)
            return RX_ERR_NULL;
    for (int j = 0; j < nsrc; ++j)
        if (!element_aligned(srcs[j], dtype))
            return RX_ERR_ALIGN;
    const void* data[] = {residual, gate, w_post, w_pre, out_h, out_z};
    for (const void* p : data)
        if (!element_aligned(p, dtype))
            return RX_ERR_ALIGN;
    if (!aligned4(rstd_post) || !aligned4(rstd_pre))
        return RX_ERR_ALIGN;
    if (rows == 0 || hidden == 0)
        return RX_OK;
    NormArgs a = {};
    for (int j = 0; j < nsrc; ++j)
        a.src[j] = srcs[j];
    a.residual = residual;
    a.gate = gate;
    a.w_post = w_post;
    a.w_pre = w_pre;
    a.out_h = out_h;
    a.out_z = out_z;
    a.rstd_post = rstd_post;
    a.rstd_pre = rstd_pre;
    a.ld_src = ld_src;
    a.ld_residual = ld_residual;
    a.ld_h = ld_h;
    a.ld_z = ld_z;
    a.rows = rows;
    a.hidden = hidden;
    a.gate_rows = gate_rows_or_one(gate_rows, rows);
    a.residual_scale = residual_scale;
    a.eps = eps;
    a.inv_hidden = (float)(1.0 / (double)hidden);
    a.nsrc = nsrc;
    return launched(launch_norm(a, dt_index(dtype), stream));
}

size_t rx_residual_norm_backward_workspace(size_t rows, size_t hidden, size_t gate_rows)
{
    if (rows > kMaxRows || hidden > (size_t)kMaxNormHidden)
        return 0;
    return norm_backward_parts(rows, hidden, gate_rows_or_one(gate_rows, rows)) * hidden * 4 * sizeof(float);
}

rx_status_t rx_residual_norm_backward(const void* const* srcs, int nsrc, size_t ld_src, const void* residual,
                                      size_t ld_residual, const void* gate, size_t gate_rows, const void* w_post,
                                      const void* w_pre, const float* rstd_post, const float* rstd_pre,
                                      float residual_scale, size_t rows, size_t hidden, rx_dtype_t dtype,
                                      const void* d_h, size_t ld_d_h, const void* d_z, size_t ld_d_z, void* d_src,
                                      size_t ld_d_src, void* d_residual, size_t ld_d_residual, float* d_gate,
                                      float* d_w_post, float* d_w_pre, void* workspace, size_t workspace_bytes,
                                      hipStream_t stream)
{
    const bool empty = rows == 0 || hidden == 0;   // no data: its pointers may be NULL
    if (!srcs || (!empty && (!d_src || (d_z && (!w_pre || !rstd_pre)) || (w_post && !rstd_post))))
        return RX_ERR_NULL;
    if (nsrc < 1 || nsrc > RX_MAX_SRC || rows > kMaxRows || hidden > (size_t)kMaxNormHidden ||
        bad_ld(ld_src, hidden, rows) || (residual && bad_ld(ld_residual, hidden, rows)) ||
        (d_h && bad_ld(ld_d_h, hidden, rows)) || (d_z && bad_ld(ld_d_z, hidden, rows)) ||
        bad_ld(ld_d_src, hidden, rows) || (d_residual && bad_ld(ld_d_residual, hidden, rows)) ||
        (gate && gate_rows < 1) || (!empty && d_residual && !residual) || (!empty && d_gate && !gate) || (!empty && d_w_post && !w_post) ||
        (!empty && d_w_pre && !w_pre) || !isfinite(residual_scale))
        return RX_ERR_ARG;
    if (!hp_type(dtype))
        return RX_ERR_DTYPE;
    for (int j = 0; j < nsrc; ++j)
        if (!srcs[j] && !empty)
            return RX_ERR_NULL;
    for (int j = 0; j < nsrc; ++j)
        if (!element_aligned(srcs[j], dtype))
            return RX_ERR_ALIGN;
    const void* data[] = {residual, gate, w_post, w_pre, d_h, d_z, d_src, d_residual};
    for (const void* p : data)
        if (!element_aligned(p, dtype))
            return RX_ERR_ALIGN;
    const void* f32[] = {rstd_post, rstd_pre, d_gate, d_w_post, d_w_pre};
    for (const void* p : f32)
        if (!aligned4(p))
            return RX_ERR_ALIGN;
    const size_t need = rx_residual_norm_backward_workspace(rows, hidden, gate_rows);
    if (need) {
        if (!workspace)
            return RX_ERR_NULL;
        if (!aligned16(workspace))
            return RX_ERR_ALIGN;
        if (workspace_bytes < need)
            return RX_ERR_ARG;
    }
    if (hidden == 0)
        return RX_OK;
    NormBwdArgs a = {};
    for (int j = 0; j < nsrc; ++j)
        a.src[j] = srcs[j];
    a.residual = residual;
    a.gate = gate;
    a.w_post = w_post;
    a.w_pre = d_z || d_w_pre ? w_pre : nullptr;
    a.rstd_post = rstd_post;
    a.rstd_pre = rstd_pre;
    a.d_h = d_h;
    a.d_z = d_z;
    a.d_src = d_src;
    a.d_residual = d_residual;
    a.d_gate = d_gate;
    a.d_w_post = d_w_post;
    a.d_w_pre = d_w_pre;
    a.ld_src = ld_src;
    a.ld_residual = ld_residual;
    a.ld_d_h = ld_d_h;
    a.ld_d_z = ld_d_z;
    a.ld_d_src = ld_d_src;
    a.ld_d_residual = ld_d_residual;
    a.rows = rows;
    a.hidden = hidden;
    a.gate_rows = gate_rows_or_one(gate_rows, rows);
    a.part_post = static_cast<float*>(workspace);
    a.residual_scale = residual_scale;
    a.inv_hidden = (float)(1.0 / (double)hidden);
    a.nsrc = nsrc;
    return launched(launch_norm_backward(a, dt_index(dtype), stream));
}

rx_status_t rx_quant_i8(const void* x, size_t ld_x, size_t rows, size_t k, rx_dtype_t dtype, void* codes,
                        size_t ld_codes, float* scales, hipStream_t stream)
{
    if (rows > 0 && (!scales || (k > 0 && (!x || !codes))))
        return RX_ERR_NULL;
    if (rows > kMaxRows || k > kMaxHidden || bad_ld(ld_x, k, rows) || bad_ld(ld_codes, k, rows))
        return RX_ERR_ARG;
    if (!hp_type(dtype))
        return RX_ERR_DTYPE;
    if (!element_aligned(x, dtype) || !aligned4(scales))
        return RX_ERR_ALIGN;
    if (rows == 0)
        return RX_OK;
    QuantI8Args a = {};
    a.x = x;
    a.codes = codes;
    a.scales = scales;
    a.ld_x = ld_x;
    a.ld_codes = ld_codes;
    a.rows = rows;
    a.k = k;
    return launched(launch_quant_i8(a, dt_index(dtype), stream));
}

rx_status_t rx_gemm_i8(const void* a, size_t ld_a, const float* a_scales, const void* b, size_t ld_b,
                       size_t stride_b, const float* b_scales, const int* offsets, int experts, size_t rows, size_t n,
                       size_t k, void* out, size_t ld_out, rx_dtype_t out_dtype, hipStream_t stream)
{
    if (rows > 0 && n > 0 && (!out || !a_scales || !b_scales || (k > 0 && (!a || !b))))
        return RX_ERR_NULL;
    const size_t k16 = (k + 15) / 16 * 16;
    if (rows > kMaxRows || n >= ((size_t)1 << 31) || k > 131071 || experts < 1 || experts > kMaxExperts ||
        (!offsets && experts != 1) || (rows > 1 && ld_a >= kMaxGemmLd) ||
        (n > 1 && ld_b >= kMaxGemmLd) || bad_ld(ld_a, k16) || bad_ld(ld_b, k16) || bad_ld(ld_out, n, rows) ||
        stride_b > kMaxLd * 16)
        return RX_ERR_ARG;
    if (!hp_type(out_dtype))
        return RX_ERR_DTYPE;
    if (!aligned16(a) || !aligned16(b) || ld_a % 16 || ld_b % 16 || stride_b % 16 || !aligned4(a_scales) ||
        !aligned4(b_scales) || !aligned4(offsets) || !element_aligned(out, out_dtype))
        return RX_ERR_ALIGN;
    // 256 x 256 outputs of 512 threads, a partial tile for every expert: a launch's limit of 2^32 threads
    if ((rows / 256 + (size_t)experts + 1) * ((n + 255) / 256) >= ((size_t)1 << 23) - 16)
        return RX_ERR_ARG;
    if (rows == 0 || n == 0)
        return RX_OK;
    GemmI8Args g = {};
    g.a = static_cast<const int8_t*>(a);
    g.b = static_cast<const int8_t*>(b);
    g.a_scales = a_scales;
    g.b_scales = b_scales;
    g.offsets = offsets;
    g.out = out;
    g.ld_a = ld_a;
    g.ld_b = ld_b;
    g.stride_b = stride_b;
    g.ld_out = ld_out;
    g.rows = (uint32_t)rows;
    g.n = (uint32_t)n;
    g.k = (uint32_t)k;
    g.experts = experts;
    return launched(launch_gemm_i8(g, dt_index(out_dtype), stream));
}

}  // extern "C"
