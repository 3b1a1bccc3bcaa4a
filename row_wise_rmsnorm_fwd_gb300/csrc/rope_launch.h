// rope_launch.h -- parameter block and kernel getters of rotary positions with head
// norms (include/rmsnorm_rope.h).  Internal to the library.
#pragma once
#include "launch.h"

namespace rmsnorm {

// A view [batch, seq, heads, head_dim]: strides in elements.
struct RopeView {
    void* p;
    int64_t batch, token, head;
};

struct RopeHeads {
    RopeView x, dy, out;
    const void* w;         // null: ones
    float* dw;             // null: not wanted
    int32_t heads;         // 0: absent
};

// Everything a kernel of this family needs; passed by value.
struct RopeParams {
    RopeHeads t[2];        // q, k
    const uint64_t* freqs;
    const void* positions; // null: the token's number in its sequence
    int64_t n_positions;
    int64_t start;
    int64_t seq;
    int64_t tokens;        // batch * seq
    float* part;           // partial sums of dw: of q (0) and k (1), part_n[i] of them from
    int64_t part_at[2];    // part + part_at[i] on, part_stride apart
    int32_t part_n[2];
    int32_t part_stride;
    int32_t lanes;         // vector kernel: lanes per head (a power of two)
    int32_t units;         // pairs of vectors per head, at most lanes
    int32_t q_ctas;        // CTAs that work on q, the others on k
    int32_t split[2];      // warps that share a token's heads of q, of k
    int32_t share[2];      // lane groups of a warp that work on one token (a power of two)
    int32_t wide;          // positions are 64-bit
    int32_t dim;
    int32_t rot;
    int32_t norm;
    float inv_dim;
    float eps;
    float mscale;
};

using RopeFn = void (*)(RopeParams);

// A warp per head, any head_dim and alignment.  back: the rotation's transpose, and with
// p.norm the norm's gradient.
RopeFn rope_any_ptr(int dtype, bool interleaved, bool back);
constexpr int kRopeAnyWarps = 4;
// Heads in vectors of vb bytes, a few lanes per head: forward, backward without a norm, and
// with one.  lanes: those of heads that are whole units for each of them, else 0.
enum : int { kRopeTurn, kRopeTurnBack, kRopeGrad };
RopeFn rope_vec_f32_turn(int vb, bool interleaved, int lanes);
RopeFn rope_vec_bf16_turn(int vb, bool interleaved, int lanes);
RopeFn rope_vec_f32_back(int vb, bool interleaved, int lanes);
RopeFn rope_vec_bf16_back(int vb, bool interleaved, int lanes);
RopeFn rope_vec_f32_grad(int vb, bool interleaved, int lanes);
RopeFn rope_vec_bf16_grad(int vb, bool interleaved, int lanes);
constexpr int kRopeVecWarps = 4;
// Sums of the parts: grid (columns / 32, 2).
RopeFn rope_reduce_ptr();
constexpr int kRopeReduceThreads = 1024;
constexpr int kRopeMaxDim = 1024;

}  // namespace rmsnorm
