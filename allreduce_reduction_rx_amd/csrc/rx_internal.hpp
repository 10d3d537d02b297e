// rx_internal.hpp -- host-side declarations shared by the entry points
// (api.hip) and the kernel translation units. Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rx {

constexpr int kMaxSrc = 16;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 64;
constexpr int kMaxNormHidden = 32768;

// Kernel arguments are passed by value, so the pointer tables travel in the
// kernarg segment and the caller's host arrays can be freed on return.
struct FlatArgs {
    const void* src[kMaxSrc];
    void* dst;
    size_t count;     // elements
};

struct TreeArgs {
    const void* src[kMaxSrc];
    void* dst[kMaxSrc];
    size_t lo, hi;    // element range of this rank's chunk
};

struct QuantArgs {
    const void* src[kMaxSrc];
    void* codes[kMaxSrc];
    float* scales[kMaxSrc];
    size_t count;     // elements per source
    int nsrc;
};

struct DrrArgs {
    const void* codes[kMaxSrc];
    const float* scales[kMaxSrc];
    void* out_codes[kMaxSrc];    // REQUANT: nout code buffers (message-indexed)
    float* out_scales[kMaxSrc];  // REQUANT: nout scale buffers (block-indexed)
    void* out_hp;                // SUM: required; REQUANT: optional
    void* out_hps[kMaxSrc];      // REQUANT to every rank's buffer: N outputs
    size_t lo, hi;               // element range processed; lo is a block multiple
    int nout;                    // REQUANT: destinations that receive the result
    int block;                   // elements per scale block
    int hp_bf16;                 // out_hp element type: 1 = BF16, 0 = FP32
    int xcd_ranges;              // 0: plain order; 1: each XCD takes a contiguous
                                 // range of workgroups; R > 1: one tile per 64-thread
                                 // workgroup, XCD x takes tiles [x R, x R + R)
};

struct AllreduceLpArgs {
    void* buf[kMaxSrc];          // the ranks' buffers, read and overwritten
    size_t count;                // elements per buffer
    int xcd_ranges;              // 1: each XCD takes a contiguous range of tiles
};

// Launch geometry helper: number of compute units of the current device
// (cached per device on first use).
int device_cu_count();

struct DispatchArgs {
    const int* ids;              // tokens x topk
    int* offsets;                // experts + 1
    int* order;                  // pairs
    int* slots;                  // pairs
    const void* x;
    void* rows;
    float* row_scales;
    uint32_t* counts;            // workspace: segments x experts
    size_t ld_x, ld_rows;        // elements
    size_t hidden;
    uint32_t tokens, pairs;
    uint32_t segment, segments;  // pairs of a counting segment, their number
    uint32_t split_vecs;         // vectors of a row one workgroup handles
    int topk, first, experts;
};

// The most pairs that one launch counts for every token, and that need no
// workspace (moe.hip).
constexpr size_t kDispatchCountAll = 4096;

struct CombineArgs {
    const void* rows;
    const int* slots;
    const float* weights;        // NULL: ones
    void* out;
    size_t ld_rows, ld_out, nrows, tokens, hidden;
    size_t chunks;               // wave units of one token
    int topk;
};

struct CombineBwdArgs {
    const void* d_out;
    const void* rows;
    const int* slots;
    const float* weights;        // NULL: ones
    const int* kept;
    void* d_rows;
    float* d_weights;            // NULL: not wanted
    size_t ld_d_out, ld_rows, ld_d_rows, nrows, tokens, hidden;
    int topk;
};

struct NormArgs {
    const void* src[kMaxSrc];
    const void* residual;
    const void* gate;
    const void* w_post;
    const void* w_pre;
    void* out_h;
    void* out_z;
    float* rstd_post;
    float* rstd_pre;
    size_t ld_src, ld_residual, ld_h, ld_z;
    size_t rows, hidden, gate_rows;
    float residual_scale, eps, inv_hidden;
    int nsrc;
};

struct NormBwdArgs {
    const void* src[kMaxSrc];
    const void* residual;
    const void* gate;
    const void* w_post;
    const void* w_pre;
    const float* rstd_post;
    const float* rstd_pre;
    const void* d_h;
    const void* d_z;
    void* d_src;
    void* d_residual;
    float* d_gate;
    float* d_w_post;
    float* d_w_pre;
    float* part_post;            // workspace (the launch lays out the parts): parts x hidden
    float* part_pre;             // workspace: parts x hidden
    float* part_gate;            // workspace: parts x 2 x hidden
    size_t ld_src, ld_residual, ld_d_h, ld_d_z, ld_d_src, ld_d_residual;
    size_t rows, hidden, gate_rows;
    size_t part_rows;            // rows of one workgroup
    size_t parts;                // workgroups
    float residual_scale, inv_hidden;
    int nsrc;
};

struct QuantI8Args {
    const void* x;
    void* codes;
    float* scales;
    size_t ld_x, ld_codes, rows, k;
};

struct GemmI8Args {
    const int8_t* a;
    const int8_t* b;
    const float* a_scales;
    const float* b_scales;
    const int* offsets;          // NULL: one matrix for all rows
    void* out;
    size_t ld_a, ld_b, stride_b, ld_out;
    uint32_t rows, n, k;
    int experts;
};

// How a kernel spreads `threads` work items (one per 16-byte vector, or 64
// per wave tile) over the GPU. Decode-size jobs (`small`) get one work item
// per thread in `wg_small`-thread workgroups, so that even a 512 KiB message
// reaches every CU; large jobs use `wg_large` threads and at most
// `max_wgs_per_cu` workgroups per CU with a grid-stride loop (fewer waves in
// flight keep the HBM access window narrow).
struct LaunchPolicy {
    unsigned wg_small;
    unsigned wg_large;
    unsigned max_wgs_per_cu;
};

// Jobs below this many threads per CU count as decode-size.
constexpr size_t kSmallThreadsPerCu = 512;

// Quantizer and dequant-reduce-requant: below this many large-variant wave
// tiles per CU a message counts as decode-size and takes the narrow variant.
constexpr size_t kSmallTilesPerCu = 8;

void launch_geometry(size_t threads, bool small, const LaunchPolicy& p, dim3& grid, dim3& block);

// RX_DEBUG=1 in the environment (read once): every launch prints its
// kernel, grid and workgroup size to stderr before it is launched.
bool debug_enabled();
hipError_t launch_logged(const char* what, const void* fn, dim3 grid, dim3 block, void** params,
                         hipStream_t s);

// Launchers (return the hipError_t of the launch). dtype: 0 FP32, 1 BF16.
// fmt: 0 E4M3, 1 E5M2.
hipError_t launch_reduce_flat(const FlatArgs& a, int nsrc, int dtype, hipStream_t s);
hipError_t launch_tree(const TreeArgs& a, int nsrc, int dtype, hipStream_t s);
hipError_t launch_quant(const QuantArgs& a, int src_dtype, int fmt, int block, hipStream_t s);
hipError_t launch_drr(const DrrArgs& a, int nsrc, int fmt, bool requant, hipStream_t s);
// One-pass low-precision allreduce of the ranks' buffers (block <= 64
// 16-byte vectors: allreduce_lp_fits), block 32..512.
bool allreduce_lp_fits(int dtype, int block);
hipError_t launch_allreduce_lp(const AllreduceLpArgs& a, int nsrc, int dtype, int fmt, int block,
                               hipStream_t s);


// The operators around a block's allreduce.
uint32_t dispatch_segment(size_t pairs);
// out: 0 the plan alone, 1 rows copied, 2 rows quantized to INT8
hipError_t launch_dispatch(const DispatchArgs& a, int dtype, int out, hipStream_t s);
hipError_t launch_combine(const CombineArgs& a, int dtype, hipStream_t s);
hipError_t launch_combine_backward(const CombineBwdArgs& a, int dtype, hipStream_t s);
hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s);
size_t norm_backward_parts(size_t rows, size_t hidden, size_t gate_rows);
hipError_t launch_norm_backward(const NormBwdArgs& a, int dtype, hipStream_t s);
hipError_t launch_quant_i8(const QuantI8Args& a, int dtype, hipStream_t s);
hipError_t launch_gemm_i8(const GemmI8Args& a, int out_dtype, hipStream_t s);

}  // namespace rx
