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
    float2* row_stats;     // three-kernel backward: a pair of sums per row
    float* part_w;         // backward: [parts][hidden] partial sums of dw (null: not wanted)
    float* part_b;         // the same for db
    float* dw;
    float* db;
    int64_t rows;
    int64_t rows_per_part; // three-kernel backward: rows of one partial sum
    int32_t hidden;
    int32_t nvec;          // vectors per row
    int32_t parts;
    int32_t group;         // staged kernels: threads per row
    int32_t rows_per_cta;  // rows of a block
    int32_t nslots;        // ring slots
    int32_t row_slot;      // bytes of a row in them
    int32_t period;        // rows after which the rows' alignment repeats
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
// Rows staged in shared memory; shift: rows of any length (see k_blockring.cuh).
NormFn layernorm_staged_ptr(int dtype, bool shift);
// Backward in three kernels: a pair of sums for each row, then dx and the
// partial column sums, then the sums over the parts.  layer: layer norm, else
// RMSNorm.
NormFn norm_bwd_rows_ptr(int dtype, int vb, bool layer);
int norm_bwd_rows_block();
NormFn norm_bwd_cols_ptr(int dtype, int vb, bool layer);
int norm_bwd_cols_block();
// One pass over staged rows, elems (16 or 32) elements per thread and row; mode:
// 0 whole vectors only and weights given (not layer norm with 32 elements), 1
// aligned rows, 2 rows of any length; rows = rows of a thread between barriers (2:
// 16 elements and mode 0, layer norm bf16 mode 1 too).
NormFn norm_bwd_staged_ptr_f32(int elems, bool layer, int rows, int mode);
NormFn norm_bwd_staged_ptr_bf16(int elems, bool layer, int rows, int mode);
constexpr int kNormBwdMaxThreads = 512;
// The last kernel, `width` (4 or 1) columns to a thread, kNormReduceCols threads
// side by side.
NormFn norm_bwd_reduce_ptr(int width);
constexpr int kNormReduceThreads = 256;
constexpr int kNormReduceCols = 8;

}  // namespace rmsnorm
