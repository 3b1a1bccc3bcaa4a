/*
 * rmsnorm_block.h -- C ABI of the boundary between two blocks of a residual
 * network: the norm behind a block's branch, its gate, the scales of branch and
 * residual, and the norm before the next block, forward and backward (same
 * library, same status codes and conventions as rmsnorm.h).
 *
 * For every row r of row-major matrices with `hidden` columns H, a branch x and
 * the residual stream it is added to, with m(.) the mean over a row:
 *
 *     n = x * rsqrt(m(x^2) + post_eps) * post_w          (post_norm = 0: n = x)
 *     h = residual_scale * residual + branch_scale * gate * n
 *     y = h * rsqrt(m(h^2) + pre_eps) * pre_w            (pre_norm = 0: no y)
 *
 * The gate has one row for every `gate_rows` rows: row r takes gate row r / gate_rows
 * (gate_rows >= rows: a learned gate for each channel; the tokens of a sequence:
 * a gate for each sequence; 1: a gate for each element).
 *
 * Given dy = dL/dy and dh, what comes to h from everything else that reads it:
 *
 *     D         = dh + the gradient of y's norm with respect to h
 *     dresidual = residual_scale * D
 *     dx        = the gradient of n's norm, from branch_scale * D * gate * post_w
 *     dpre_w[j]    = sum_r dy * h * rsqrt(m(h^2) + pre_eps)
 *     dpost_w[j]   = branch_scale * sum_r D * gate * x * rsqrt(m(x^2) + post_eps)
 *     dgate[s, j]  = branch_scale * sum over the rows of gate row s of D * n
 *
 * fp32 arithmetic for both types: bf16 inputs are widened exactly, y is formed
 * from the h that has not been rounded yet, every output is rounded once.  The
 * backward pass takes the h that the forward pass wrote, and both norms' factors
 * are computed again from h and x.  Gradients of weights and gate are fp32.
 *
 *  - x, residual, h, y, dy, dh, dx, dresidual: DEVICE pointers, rows*hidden
 *    elements, contiguous row-major; post_w, pre_w: hidden elements of the same
 *    type, NULL for ones; gate: max(1, ceil(rows / gate_rows)) * hidden elements,
 *    NULL for ones; dpost_w, dpre_w: hidden floats, dgate: one for each element of
 *    the gate.  Any element alignment.
 *  - y must be given with pre_norm and be NULL without; so must dy, and h then is not
 *    read by the backward pass and may be NULL.  dh may be NULL: zeros.
 *    dpost_w, dpre_w and dgate may each be NULL: not computed; they must be NULL where
 *    there is no such norm or gate.
 *  - An output may be one of the inputs of rows*hidden elements (in place); any
 *    other overlap of an output or the workspace with another argument is rejected.
 *  - rows >= 0; 1 <= hidden <= 2^20; gate_rows >= 1 if there is a gate; scales finite;
 *    eps finite and >= 0.  rows == 0: OK; the backward pass then writes zeros to
 *    dpost_w, dpre_w and the one row of dgate.
 *  - Asynchronous on `stream`, allocating nothing; kernels are launched as
 *    rmsnorm.h's common contract states.  Argument errors are found on the host
 *    before any launch.  Results are bitwise repeatable on a device: sums have
 *    a fixed order, without atomics.
 *  - workspace: 16-byte aligned device memory of at least the bytes that
 *    rmsnorm_block_bwd_workspace gives (a few MB, and 8 bytes for each element of a
 *    gate of several rows), contents undefined before and after.  It is
 *    in use until the call's kernels have run, so calls that can overlap on the
 *    GPU (other streams, two captured graphs) need one each.
 */
#ifndef RMSNORM_BLOCK_H_
#define RMSNORM_BLOCK_H_

#include "rmsnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    const void* post_w;      /* device, or NULL: ones */
    const void* pre_w;
    const void* gate;        /* device, or NULL: ones */
    int64_t gate_rows;       /* rows that share a row of the gate */
    float residual_scale;
    float branch_scale;
    float post_eps;
    float pre_eps;
    int32_t post_norm;       /* 1: the branch is normed */
    int32_t pre_norm;        /* 1: y is wanted */
} rmsnorm_block_t;

/* h and, with pre_norm, y. */
rmsnorm_status_t rmsnorm_block_fwd_f32(const float* x, const float* residual, float* h, float* y,
                                       int64_t rows, int64_t hidden, const rmsnorm_block_t* block,
                                       rmsnorm_stream_t stream);

/* The same for bfloat16 arrays, weights and gate (raw 16-bit patterns). */
rmsnorm_status_t rmsnorm_block_fwd_bf16(const uint16_t* x, const uint16_t* residual, uint16_t* h,
                                        uint16_t* y, int64_t rows, int64_t hidden,
                                        const rmsnorm_block_t* block, rmsnorm_stream_t stream);

/* Either dtype, with options (`opt` may be NULL): opt->path RMSNORM_PATH_AUTO,
 * RMSNORM_PATH_STAGED (rows staged in shared memory by bulk copies, read from HBM once: x and
 * residual, backward dy, dh, x and h, on 16-byte boundaries; if rows, weights, gate and
 * outputs are multiples of 16 bytes on such boundaries too, rows of at most 512 KB, backward
 * 256 KB, split over a thread-block cluster above 32 KB, backward 16 KB, which
 * opt->cluster = 2, 4, 8 or 16 forces; else rows of 16 bytes to 24 KB, backward 16 KB;
 * RMSNORM_ERR_UNSUPPORTED otherwise), RMSNORM_PATH_ROWREG (forward; rows held in registers, at
 * most 8192 vectors of 2, 4 or 8 bytes: what one of those is the widest for; else
 * RMSNORM_ERR_UNSUPPORTED) or RMSNORM_PATH_TWOPASS (a CTA per row that reads it again for each
 * sum: any width and alignment); opt->wait_timeout_ns; and in the test build of the library
 * opt->fault_inject with RMSNORM_PATH_STAGED: 1 = each CTA's first copy is withheld, 2 =
 * with opt->cluster, rank 0's first sums are, 3 = with opt->cluster, the wait of rank 0's last
 * thread for the first sums counts as run out (elsewhere RMSNORM_ERR_UNSUPPORTED; 3 without the
 * test build RMSNORM_ERR_INVALID_ARG).  Every other field but epilogue_alpha, which is not read,
 * must be zero, else RMSNORM_ERR_INVALID_ARG. */
rmsnorm_status_t rmsnorm_block_fwd_ex(int32_t dtype, const void* x, const void* residual, void* h,
                                      void* y, int64_t rows, int64_t hidden,
                                      const rmsnorm_block_t* block, const rmsnorm_options_t* opt,
                                      rmsnorm_stream_t stream);

/* Bytes of workspace that a backward pass of this shape takes on the current
 * device, whatever the pointers (of `block`, gate is looked at for NULL, and
 * gate_rows). */
rmsnorm_status_t rmsnorm_block_bwd_workspace(int32_t dtype, int64_t rows, int64_t hidden,
                                             const rmsnorm_block_t* block, size_t* bytes);

/* dx, dresidual and the gradients of weights and gate that are wanted. */
rmsnorm_status_t rmsnorm_block_bwd_f32(const float* dy, const float* dh, const float* x,
                                       const float* h, float* dx, float* dresidual, float* dpost_w,
                                       float* dpre_w, float* dgate, int64_t rows, int64_t hidden,
                                       const rmsnorm_block_t* block, void* workspace,
                                       size_t workspace_bytes, rmsnorm_stream_t stream);

/* The same for bfloat16 arrays, weights and gate; dpost_w, dpre_w and dgate are fp32. */
rmsnorm_status_t rmsnorm_block_bwd_bf16(const uint16_t* dy, const uint16_t* dh, const uint16_t* x,
                                        const uint16_t* h, uint16_t* dx, uint16_t* dresidual,
                                        float* dpost_w, float* dpre_w, float* dgate, int64_t rows,
                                        int64_t hidden, const rmsnorm_block_t* block,
                                        void* workspace, size_t workspace_bytes,
                                        rmsnorm_stream_t stream);

/* Either dtype, with options as for rmsnorm_block_fwd_ex (no RMSNORM_PATH_ROWREG;
 * RMSNORM_PATH_TWOPASS: the
 * sums of each row, then the outputs and partial column sums, each reading the arrays
 * once: any width and alignment). */
rmsnorm_status_t rmsnorm_block_bwd_ex(int32_t dtype, const void* dy, const void* dh, const void* x,
                                      const void* h, void* dx, void* dresidual, float* dpost_w,
                                      float* dpre_w, float* dgate, int64_t rows, int64_t hidden,
                                      const rmsnorm_block_t* block, void* workspace,
                                      size_t workspace_bytes, const rmsnorm_options_t* opt,
                                      rmsnorm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RMSNORM_BLOCK_H_ */
