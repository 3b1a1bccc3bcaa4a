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
    float* part;           // partial sums of dw, [parts][2][dim]
    int32_t parts;
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
// Sums of the parts: grid (columns / 32, 2).
RopeFn rope_reduce_ptr();
constexpr int kRopeReduceThreads = 1024;
constexpr int kRopeMaxDim = 1024;

}  // namespace rmsnorm
