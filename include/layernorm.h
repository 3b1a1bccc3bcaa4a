/*
 * layernorm.h -- C ABI of librmsnorm's layer norm, forward and backward (same
 * library, same status codes and conventions as rmsnorm.h).
 *
 * For every row r of a row-major matrix x with `hidden` columns H:
 *
 *     mean[r] = (1/H) * sum_j x[r,j]
 *     rstd[r] = rsqrt((1/H) * sum_j (x[r,j] - mean[r])^2 + eps)
 *     y[r,j]  = (x[r,j] - mean[r]) * rstd[r] * w[j] + b[j]
 *
 * and, given dy = dL/dy, with xh = (x - mean) * rstd, g = dy * w and m(.) the
 * mean over a row:
 *
 *     dx[r,j] = rstd[r] * (g[r,j] - m(g)[r] - xh[r,j] * m(g * xh)[r])
 *     dw[j]   = sum_r dy[r,j] * xh[r,j]          db[j] = sum_r dy[r,j]
 *
 * fp32 arithmetic for both types (bf16 inputs are widened exactly, y and dx are
 * rounded once); the variance is taken about the mean, never as a difference of
 * large sums.  dw and db are fp32 for both types, as an optimiser's master
 * copy wants them.  A NaN or an infinity in a row of x makes that row of y and dx,
 * and with it dw, NaN; db, the sum of dy alone, is not touched by it.
 *
 *  - x, dy, y, dx: DEVICE pointers, rows*hidden elements, contiguous row-major;
 *    w, b: hidden elements of the same type, NULL for ones and zeros; mean,
 *    rstd: rows floats; dw, db: hidden floats.  Any element alignment.
 *  - y == x, and dx == dy or dx == x, are allowed (in place); any other overlap
 *    of an output or the workspace with another argument is rejected.
 *  - rows >= 0; 1 <= hidden <= 2^31-1; eps finite and >= 0.  rows == 0: OK;
 *    the backward pass then writes zeros to dw and db.
 *  - Asynchronous on `stream`, allocating nothing; kernels are launched as
 *    rmsnorm.h's common contract states.  Argument errors are found on the host
 *    before any launch.  Results are bitwise repeatable on a device: sums have
 *    a fixed order, without atomics.
 *  - workspace: 16-byte aligned device memory of at least the bytes that
 *    layernorm_bwd_workspace gives, contents undefined before and after.  It is
 *    in use until the call's kernels have run, so calls that can overlap on the
 *    GPU (other streams, two captured graphs) need one each.
 */
#ifndef LAYERNORM_H_
#define LAYERNORM_H_

#include "rmsnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* y, and mean and rstd for a backward pass (each may be NULL: not written). */
rmsnorm_status_t layernorm_fwd_f32(const float* x, const float* w, const float* b, float* y,
                                   float* mean, float* rstd, int64_t rows, int64_t hidden,
                                   float eps, rmsnorm_stream_t stream);

/* The same for bfloat16 x, w, b and y (raw 16-bit patterns). */
rmsnorm_status_t layernorm_fwd_bf16(const uint16_t* x, const uint16_t* w, const uint16_t* b,
                                    uint16_t* y, float* mean, float* rstd, int64_t rows,
                                    int64_t hidden, float eps, rmsnorm_stream_t stream);

/* Either dtype, with options (`opt` may be NULL): opt->path RMSNORM_PATH_AUTO,
 * RMSNORM_PATH_STAGED (rows staged in shared memory by bulk copies, read from
 * HBM once: x and y on 16-byte boundaries, rows of any length from 32 bytes (16,
 * if they, w and b are multiples of 16 bytes, on such boundaries) to what two of
 * fit shared memory, else RMSNORM_ERR_UNSUPPORTED) or RMSNORM_PATH_TWOPASS (a CTA per row that
 * reads it twice: any width and alignment); opt->wait_timeout_ns; and in the
 * test build of the library opt->fault_inject = 1 with RMSNORM_PATH_STAGED
 * (each CTA's first copy is withheld; elsewhere RMSNORM_ERR_UNSUPPORTED).
 * Every other field but epilogue_alpha, which is not read, must be zero, else
 * RMSNORM_ERR_INVALID_ARG. */
rmsnorm_status_t layernorm_fwd_ex(int32_t dtype, const void* x, const void* w, const void* b,
                                  void* y, float* mean, float* rstd, int64_t rows, int64_t hidden,
                                  float eps, const rmsnorm_options_t* opt,
                                  rmsnorm_stream_t stream);

/* Bytes of workspace that a backward pass of this shape takes on the current
 * device, whatever the pointers' alignment. */
rmsnorm_status_t layernorm_bwd_workspace(int32_t dtype, int64_t rows, int64_t hidden,
                                         size_t* bytes);

/* dx, dw and db from dy, the forward pass's x and w, and the mean and rstd that
 * it wrote.  dw and db may each be NULL: not computed. */
rmsnorm_status_t layernorm_bwd_f32(const float* dy, const float* x, const float* w,
                                   const float* mean, const float* rstd, float* dx, float* dw,
                                   float* db, int64_t rows, int64_t hidden, void* workspace,
                                   size_t workspace_bytes, rmsnorm_stream_t stream);

/* The same for bfloat16 dy, x, w and dx. */
rmsnorm_status_t layernorm_bwd_bf16(const uint16_t* dy, const uint16_t* x, const uint16_t* w,
                                    const float* mean, const float* rstd, uint16_t* dx, float* dw,
                                    float* db, int64_t rows, int64_t hidden, void* workspace,
                                    size_t workspace_bytes, rmsnorm_stream_t stream);

/* Either dtype, with options as for layernorm_fwd_ex.  RMSNORM_PATH_STAGED: x
 * and dy read from HBM once (x, dy and dx on 16-byte boundaries; rows as there, of
 * at most 16384 elements, in fp32 of 14400: two rows of x and dy, and rows off the
 * boundaries with the weights beside them, which ends at 11517, must fit shared
 * memory); RMSNORM_PATH_TWOPASS: a pair of sums per row, then dx and partial column
 * sums, each reading x and dy once. */
rmsnorm_status_t layernorm_bwd_ex(int32_t dtype, const void* dy, const void* x, const void* w,
                                  const float* mean, const float* rstd, void* dx, float* dw,
                                  float* db, int64_t rows, int64_t hidden, void* workspace,
                                  size_t workspace_bytes, const rmsnorm_options_t* opt,
                                  rmsnorm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LAYERNORM_H_ */
