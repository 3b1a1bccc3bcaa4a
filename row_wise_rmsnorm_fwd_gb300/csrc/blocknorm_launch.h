// blocknorm_launch.h -- parameter block and kernel getters of the boundary between
// two blocks (include/rmsnorm_block.h).  Internal to the library.
#pragma once
#include "launch.h"

namespace rmsnorm {

// Failure injection of this family beside common.cuh's, in the test build only: one thread takes
// its wait for a cluster's sums as run out.
constexpr int kFaultClusterLateThread = 3;

// Everything a kernel of this family needs; passed by value.
struct BlockParams {
    const void* x;
    const void* residual;  // forward
    const void* dy;        // backward
    const void* dh;        // null: zeros
    const void* h_in;      // backward: the forward pass's h
    const void* post_w;    // null: ones
    const void* pre_w;
    const void* gate;
    void* h;               // forward outputs; y null: not wanted
    void* y;
    void* dx;              // backward outputs
    void* dres;
    float4* row_stats;     // any-width backward: the four factors of each row
    float* part_pre;       // partial sums of dpre_w (null: not wanted)
    float* part_gate;      // partial sums of D * xh, from which dpost_w and dgate are made
    float* gate_sums;      // [gates][hidden], their sums (several gate rows and dpost_w)
    float* dpost_w;
    float* dpre_w;
    float* dgate;
    int64_t rows;
    int64_t gate_rows;     // rows of a gate row; without a gate: rows
    int64_t gates;         // rows of the gate, 1 without one
    int64_t rows_per_part; // any-width backward: rows of a part
    int64_t parts_per_gate;
    int64_t parts;         // any-width backward: gates * parts_per_gate
    int64_t units;         // staged backward: CTAs or clusters, unit u's sums of gate row s
                           // being part u + s; 0: the parts are the any-width kernel's
    int32_t pre_parts;     // parts of dpre_w
    int32_t few_parts;     // several gate rows of few parts each
    int32_t hidden;
    int32_t nvec;          // vectors per row
    // staged kernels
    int64_t blocks;        // blocks of rows, of all gate rows
    int64_t blocks_per_gate;
    int32_t block_rows;    // rows of a block: row groups of a CTA
    int32_t group;         // threads per row (cluster > 1: per slice)
    int32_t cluster;       // CTAs per row
    int32_t slice_vecs;    // vectors of a CTA's slice of a row
    int32_t nslots;        // ring slots
    int32_t row_slot;      // ragged rows: bytes of a row in a slot
    int32_t fault;         // failure-detection test builds only (else always 0)
    unsigned* status;
    uint64_t timeout_ns;
    int32_t post;          // the branch is normed
    int32_t pre;           // y is wanted
    float inv_hidden;
    float residual_scale;
    float branch_scale;
    float post_eps;
    float pre_eps;
};

using BlockFn = void (*)(BlockParams);

// dtype: 0 = fp32, 1 = bf16; vb = bytes per vector.  Any width.
BlockFn blocknorm_fwd_any_ptr(int dtype, int vb);
// Rows of vectors of less than 16 bytes, nv = kBlockRegsVecs or twice as many to a thread.
BlockFn blocknorm_fwd_regs_ptr(int dtype, int vb, int nv);
constexpr int kBlockRegsVecs = 4;
constexpr int kBlockRegsMaxThreads = 1024;
BlockFn blocknorm_bwd_rows_ptr(int dtype, int vb);
BlockFn blocknorm_bwd_cols_ptr(int dtype, int vb);
int blocknorm_rows_block();
int blocknorm_cols_block();
// Sums over the parts, `width` (4 or 1) columns to a thread.  gates: one grid row (y) for
// dpre_w and one for each gate row; else dpost_w from the sums of several gate rows.
BlockFn blocknorm_reduce_ptr(int dtype, int width, bool gates);
// Rows staged in shared memory, read once.  post, pre: the norms; cluster: rows split over
// a thread-block cluster; whole: every thread has all its vectors, there are weights for
// the norms (one at least), and a gate as `gate` says.
struct BlockVariant {
    int dtype;
    int vb;               // bytes of a vector; less than 16: ragged rows
    bool back, post, pre, cluster, whole, gate;
};
BlockFn blocknorm_fwd_staged_f32(const BlockVariant& v);
BlockFn blocknorm_fwd_staged_bf16(const BlockVariant& v);
BlockFn blocknorm_bwd_staged_f32(const BlockVariant& v);
BlockFn blocknorm_bwd_staged_bf16(const BlockVariant& v);
BlockFn blocknorm_fwd_ragged_f32(const BlockVariant& v);
BlockFn blocknorm_fwd_ragged_bf16(const BlockVariant& v);
BlockFn blocknorm_bwd_ragged_f32(const BlockVariant& v);
BlockFn blocknorm_bwd_ragged_bf16(const BlockVariant& v);
constexpr int kBlockStagedBytes = 32;       // bytes of a row to a thread
constexpr int kBlockFwdMaxThreads = 1024;
constexpr int kBlockFwdRaggedMaxThreads = 768;   // their pieces take more registers
constexpr int kBlockBwdMaxThreads = 512;
constexpr int kBlockReduceThreads = 256;
constexpr int kBlockReduceCols = 8;

}  // namespace rmsnorm
