// norm_launch.h -- parameter block and kernel getters of layer norm and of the
// norm backward passes.  Internal to the library.
#pragma once
#include "launch.h"

namespace rmsnorm {

// Everything a kernel of these families needs; passed by value.
struct NormParams {
    const void* x;
    const void* dy;        // backward
    const void* w;         // null: ones
    const void* b;         // layer norm forward; null: zeros
    void* out;             // y, or dx
    float* mean;           // layer norm: written forward (null: not wanted), read backward
    float* rstd;
    float2* row_stats;     // two-kernel backward: a pair of sums per row
    float* part_w;         // backward: [parts][hidden] partial sums of dw (null: not wanted)
    float* part_b;         // the same for db
    float* dw;
    float* db;
    int64_t rows;
    int64_t rows_per_part; // two-kernel backward: rows of one partial sum
    int32_t hidden;
    int32_t nvec;          // vectors per row
    int32_t parts;
    int32_t group;         // staged kernels: threads per row
    int32_t rows_per_cta;  // rows of a block
    int32_t nslots;        // ring slots, and one array's bytes of each
    int32_t slot_bytes;
    int32_t fault;         // failure-detection test builds only (else always 0)
    unsigned* status;
    uint64_t timeout_ns;
    float inv_hidden;
    float eps;
};

using NormFn = void (*)(NormParams);

// dtype: 0 = fp32, 1 = bf16; vb = bytes per vector.
NormFn layernorm_twopass_ptr(int dtype, int vb);
int layernorm_twopass_block();
NormFn layernorm_staged_ptr(int dtype, int vb);
// Backward in three kernels: a pair of sums for each row, then dx and the
// partial column sums, then the sums over the parts.  layer: layer norm, else
// RMSNorm.
NormFn norm_bwd_rows_ptr(int dtype, int vb, bool layer);
int norm_bwd_rows_block();
NormFn norm_bwd_cols_ptr(int dtype, int vb, bool layer);
int norm_bwd_cols_block();
// One pass over staged rows, kNormBwdElems elements per thread and row: rows =
// rows of a thread between barriers (2: only if full), full: whole vectors only
// and weights given.
NormFn norm_bwd_staged_ptr_f32(int vb, bool layer, int rows, bool full);
NormFn norm_bwd_staged_ptr_bf16(int vb, bool layer, int rows, bool full);
constexpr int kNormBwdElems = 16;
constexpr int kNormBwdMaxThreads = 512;
NormFn norm_bwd_reduce_ptr();
constexpr int kNormReduceCols = 8;       // columns of one CTA of the last kernel
constexpr int kNormReduceLanes = 32;     // parts it adds side by side

}  // namespace rmsnorm
