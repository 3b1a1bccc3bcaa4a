/*
 * rmsnorm_rope.h -- C ABI of rotary positions with the norm of each head before
 * them, for the queries and keys of attention, forward and backward (same library,
 * same status codes and conventions as rmsnorm.h).
 *
 * For the D = head_dim elements v of every token and head, with m(.) their mean:
 *
 *     n = v * rsqrt(m(v^2) + eps) * w                     (norm = 0: n = v)
 *     a[i] = position * frequency[i],   0 <= i < rot_dim / 2
 *     (p, q) -> mscale * (p cos a[i] - q sin a[i],  q cos a[i] + p sin a[i])
 *
 * for the pairs (n[i], n[i + rot_dim/2]), or (n[2i], n[2i+1]) if interleaved; elements
 * from rot_dim on are n itself.  The backward pass turns dy back (the transpose: angles
 * negated, same mscale) and applies the norm's gradient; dw is the sum over all
 * tokens and heads.
 *
 * Token (b, s) stands at start + positions[(b * seq + s) mod n_positions], or, without
 * positions, at start + s.  Frequencies are 64-bit fixed-point numbers of turns per
 * position, frequency / (2 pi) * 2^64 modulo 2^64 (rmsnorm_rope_freqs): the product
 * with a 64-bit position modulo 2^64 is the angle modulo a turn, exactly.  The frequency
 * itself is rounded once, to the nearest of them (frequencies of up to 2^40 turns a position, which
 * small divisors give): it is off by 2^-65 turns, which position p makes p * 2^-65 (2^-25 at 2^40).
 *
 * fp32 arithmetic for both types: bf16 inputs are widened exactly, outputs are
 * rounded once; dw is fp32.
 *
 *  - q and k are views [batch, seq, heads, head_dim] of DEVICE memory: a pointer and the
 *    strides, in elements, of batch, token and head; the head's elements are
 *    contiguous.  They may lie inside a larger array (q, k and v of one projection) or
 *    have heads before tokens.  k may be NULL (q alone).  Any element alignment.
 *  - out may be the x (backward: the dy or the x) of its own heads: same address and
 *    strides.  Else outputs overlap nothing.  Views of q and k may interleave
 *    inside one array.
 *  - 2 <= head_dim <= 1024; rot_dim even, 2 <= rot_dim <= head_dim; heads >= 1;
 *    batch, seq >= 0 (a product of 0: OK, no launch but zeros to dw); batch * seq * heads
 *    <= 2^40; n_positions >= 1 if there are positions; eps finite and >= 0, mscale finite.
 *  - Asynchronous on `stream`, allocating nothing; kernels are launched as
 *    rmsnorm.h's common contract states.  Argument errors are found on the host
 *    before any launch.  Results are bitwise repeatable on a device.
 *  - workspace (backward with a dw): 16-byte aligned device memory of at least the
 *    bytes that rmsnorm_rope_bwd_workspace gives, contents undefined before and
 *    after; calls that can overlap on the GPU need one each.
 */
#ifndef RMSNORM_ROPE_H_
#define RMSNORM_ROPE_H_

#include "rmsnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The heads of q or of k; strides in elements, of batch, token and head. */
typedef struct {
    const void* x;              /* forward; backward: read with norm only */
    const void* dy;             /* backward */
    void* out;                  /* written: the turned heads; backward: dx */
    const void* w;              /* head_dim elements of the same type, NULL: ones */
    float* dw;                  /* backward with norm: head_dim floats, or NULL */
    int64_t heads;
    int64_t x_stride[3];
    int64_t dy_stride[3];
    int64_t out_stride[3];
} rmsnorm_rope_heads_t;

typedef struct {
    const uint64_t* freqs;      /* device, rot_dim / 2 */
    const void* positions;      /* device, or NULL */
    int64_t n_positions;
    int64_t start;
    int32_t position_bytes;     /* 4 or 8 (int32_t or int64_t), if there are positions */
    int32_t rot_dim;
    int32_t interleaved;
    int32_t norm;
    float eps;
    float mscale;
} rmsnorm_rope_t;

/* Scaling of the frequencies for contexts longer than those of training. */
typedef enum {
    RMSNORM_ROPE_NONE = 0,
    RMSNORM_ROPE_LINEAR = 1,    /* all divided by factor */
    RMSNORM_ROPE_BASE = 2,      /* base * factor^(rot_dim / (rot_dim - 2)): the slowest divided by
                                   factor, the fastest kept; rot_dim >= 4 */
    RMSNORM_ROPE_RAMP = 3,      /* by pair number: pairs that make more than `high` turns over
                                   original_len kept, fewer than `low` divided, a ramp between the
                                   two pair numbers (rounded outwards, the first at least 0, the
                                   second at most rot_dim - 1); mscale 0.1 ln(factor) + 1
                                   (Peng et al., "YaRN: Efficient Context Window Extension of Large
                                   Language Models", 2023) */
    RMSNORM_ROPE_BANDS = 4      /* by turns over original_len: `high` and more kept, `low` and fewer
                                   divided, in proportion between them */
} rmsnorm_rope_scaling_t;

typedef struct {
    double base;                /* frequency[i] = base^(-2i / rot_dim), base > 1 */
    double factor;              /* >= 1 */
    double low, high;           /* 0 < low < high, RAMP and BANDS */
    int64_t original_len;       /* >= 1, RAMP and BANDS */
    const double* divisors;     /* host, rot_dim / 2 numbers > 0 that the scaled frequencies are
                                   divided by, or NULL */
    int32_t scaling;            /* rmsnorm_rope_scaling_t */
    int32_t rot_dim;
} rmsnorm_rope_rule_t;

/* Fill `freqs` (HOST memory, rot_dim / 2) and *mscale for a rule.  Host function, no device
 * needed. */
rmsnorm_status_t rmsnorm_rope_freqs(const rmsnorm_rope_rule_t* rule, uint64_t* freqs,
                                    float* mscale);

rmsnorm_status_t rmsnorm_rope_fwd_f32(const rmsnorm_rope_heads_t* q, const rmsnorm_rope_heads_t* k,
                                      int64_t batch, int64_t seq, int64_t head_dim,
                                      const rmsnorm_rope_t* rope, rmsnorm_stream_t stream);

rmsnorm_status_t rmsnorm_rope_fwd_bf16(const rmsnorm_rope_heads_t* q,
                                       const rmsnorm_rope_heads_t* k, int64_t batch, int64_t seq,
                                       int64_t head_dim, const rmsnorm_rope_t* rope,
                                       rmsnorm_stream_t stream);

/* Either dtype, with options (`opt` may be NULL): opt->path RMSNORM_PATH_AUTO or
 * RMSNORM_PATH_TWOPASS (a warp per head that reads it twice: any head_dim, strides and
 * alignment).  Every other field but wait_timeout_ns and epilogue_alpha, which are not
 * read, must be zero, else RMSNORM_ERR_INVALID_ARG. */
rmsnorm_status_t rmsnorm_rope_fwd_ex(int32_t dtype, const rmsnorm_rope_heads_t* q,
                                     const rmsnorm_rope_heads_t* k, int64_t batch, int64_t seq,
                                     int64_t head_dim, const rmsnorm_rope_t* rope,
                                     const rmsnorm_options_t* opt, rmsnorm_stream_t stream);

/* Bytes of workspace that a backward pass with a dw takes on the current device, whatever
 * the views; `heads` of q and k together. */
rmsnorm_status_t rmsnorm_rope_bwd_workspace(int32_t dtype, int64_t batch, int64_t seq,
                                            int64_t heads, int64_t head_dim, size_t* bytes);

rmsnorm_status_t rmsnorm_rope_bwd_f32(const rmsnorm_rope_heads_t* q, const rmsnorm_rope_heads_t* k,
                                      int64_t batch, int64_t seq, int64_t head_dim,
                                      const rmsnorm_rope_t* rope, void* workspace,
                                      size_t workspace_bytes, rmsnorm_stream_t stream);

rmsnorm_status_t rmsnorm_rope_bwd_bf16(const rmsnorm_rope_heads_t* q,
                                       const rmsnorm_rope_heads_t* k, int64_t batch, int64_t seq,
                                       int64_t head_dim, const rmsnorm_rope_t* rope,
                                       void* workspace, size_t workspace_bytes,
                                       rmsnorm_stream_t stream);

/* Either dtype, with options as for rmsnorm_rope_fwd_ex. */
rmsnorm_status_t rmsnorm_rope_bwd_ex(int32_t dtype, const rmsnorm_rope_heads_t* q,
                                     const rmsnorm_rope_heads_t* k, int64_t batch, int64_t seq,
                                     int64_t head_dim, const rmsnorm_rope_t* rope, void* workspace,
                                     size_t workspace_bytes, const rmsnorm_options_t* opt,
                                     rmsnorm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RMSNORM_ROPE_H_ */
