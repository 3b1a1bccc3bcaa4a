// relbias_launch.h -- parameter block and kernel getters of the row softmax
// with a learned relative position bias.  Internal to the library.
#pragma once
#include "launch.h"

namespace rmsnorm {

constexpr int kBiasMaxBuckets = 256;
constexpr int kBiasMaxDistance = 4096;
constexpr int kBiasMaxKeys = 1 << 30;

struct BiasParams {
    const void* x;          // forward: scores; backward: dy
    const void* y;          // backward: the forward pass's outputs
    void* out;              // forward: y; backward: dx
    const void* table;      // forward: [num_buckets][heads]
    double* part;           // backward: [heads][parts][num_buckets] (null: not wanted)
    float* dtable;          // backward: [num_buckets][heads]
    const int32_t* q_start; // [batch] or null
    const int32_t* kv_len;  // [batch] or null
    int64_t q_offset;
    int64_t elems;          // of x, y and out
    float scale;
    int32_t head_rows;      // rows of one head: batch * q_len
    int32_t q_len;
    int32_t k_len;
    int32_t heads;
    int32_t nvec;           // vectors per row
    int32_t parts;          // CTAs per head
    int32_t group;          // threads per row
    int32_t rows_per_cta;
    int32_t turns;          // backward: row groups that share a window in turn
    int32_t causal;
    int32_t both;           // bidirectional: positive positions in the upper half
    int32_t num_buckets;
    int32_t half;           // buckets of one direction
    int32_t edges[kBiasMaxBuckets];   // smallest distance of each bucket of a direction
};

using BiasFn = void (*)(BiasParams);

// Floats of the window over relative positions that a kernel of `epv` elements
// per vector keeps in shared memory (see k_relbias.cuh).
constexpr int bias_window_slots(int lo, int hi, int epv) {
    const int n = lo + hi + 2 * epv;
    return n + (epv > 1 ? n / epv : 0) + 1;
}

// The same for the register kernels' window: `copies` shifted copies of it in
// chunks that a vector load takes (see k_relbias.cuh).
struct BiasVecWindow {
    int size, copies, half, copy;      // positions, copies, chunks of a half, floats of a copy
};
constexpr BiasVecWindow bias_vec_window(int lo, int hi, int epv) {
    BiasVecWindow w{};
    w.size = lo + hi + 4 * epv;
    w.copies = 4;                      // epv is 4 or 8
    const int chunks = w.size / w.copies + 1;
    w.half = (chunks + 1) / 2;
    w.copy = (epv == 8 ? 2 * w.half : chunks) * w.copies;
    return w;
}

BiasFn relbias_fwd_wide_ptr(int dtype, int vb);
BiasFn relbias_bwd_wide_ptr(int dtype, int vb);
int relbias_wide_block();
// Rows in registers: nv (4 or 6) 16-byte vectors per thread, blocks of up to kBiasMaxThreads
// threads; shift: rows that are not a multiple of 16 bytes.
BiasFn relbias_rowreg_ptr(int dtype, int nv, bool shift, bool bwd, bool turns);
constexpr int kBiasMaxThreads = 512;
BiasFn relbias_reduce_ptr();
int relbias_reduce_block();

}  // namespace rmsnorm
