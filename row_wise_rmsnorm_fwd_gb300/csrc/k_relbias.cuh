// k_relbias.cuh -- row softmax of attention scores with a learned relative
// position bias, and its backward pass.
//
// Scores x[b, h, i, j] (batch, head, query, key).  The query stands at
// q = q_offset + q_start[b] + i, so the key's relative position is r = j - q:
//     v = scale * x + t[bucket(r), h]      over the valid keys of the row,
//     y = exp(v - max v) / sum exp(v - max v),  0 at the other keys.
// Both masks, j < kv_len[b] and (causal) r <= 0, leave a prefix [0, n) of the
// row valid; nothing outside it is read, and a row with n = 0 is all zero.
//     backward: ds = y * (dy - sum_j y * dy), dx = scale * ds,
//               dt[k, h] = sum of ds over b, i and the j with bucket(r) = k.
//
// bucket(r) is constant for r <= -lo and for r >= hi (lo: the last edge of a
// direction; hi = lo, or 0 if positive positions have no buckets of their
// own), so a CTA, which works on one head, keeps the head's biases (backward:
// its sums) of the window in between, one float per relative position, in
// shared memory.  A vector of keys wholly outside the window costs one
// comparison; inside, a lookup per element.  The window is stored with one
// unused float after every EPV, so that 32 lanes reading every EPV-th
// position hit 32 banks.
//
// The sums of ds are deterministic: within a row every relative position of
// the window belongs to one thread, rows of one window pass one after the
// other, and every kBiasFoldRows rows the window is folded into one fp64 sum
// per bucket in a fixed order (which also keeps the fp32 chains short).
#pragma once
#include "k_normbwd.cuh"
#include "k_softmax.cuh"
#include "relbias_launch.h"

namespace rmsnorm {

constexpr int kBiasFoldRows = 64;

template <int EPV>
__device__ __forceinline__ int bias_slot(int idx) {
    return EPV > 1 ? idx + idx / EPV : idx;      // EPV is a power of two
}

// Buckets of one direction: the last one whose edge is at most n.
__device__ __forceinline__ int bias_bucket_of(const BiasParams& p, int n) {
    int lo = 0, hi = p.half;                     // edges[lo] <= n < edges[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.edges[mid] <= n) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int bias_bucket(const BiasParams& p, int r) {
    if (p.both) return bias_bucket_of(p, r < 0 ? -r : r) + (r > 0 ? p.half : 0);
    return bias_bucket_of(p, r < 0 ? -r : 0);
}

struct BiasWindow {
    int lo, hi;              // constant for r <= -lo and for r >= hi
    __device__ __forceinline__ explicit BiasWindow(const BiasParams& p)
        : lo(p.edges[p.half - 1]), hi(p.both ? p.edges[p.half - 1] : 0) {}
};

// One row: where it starts, its valid keys [0, n), and r of key 0.
struct BiasRow {
    int64_t at;              // element index of the row's key 0
    int n;
    int r0;
};

__device__ __forceinline__ BiasRow bias_row(const BiasParams& p, int head, int row) {
    const int b = row / p.q_len;
    const int i = row - b * p.q_len;
    BiasRow o;
    o.at = ((static_cast<int64_t>(b) * p.heads + head) * p.q_len + i) * p.k_len;
    int64_t q = p.q_offset + i;
    if (p.q_start) q += p.q_start[b];
    // positions further than this from every key change neither r's side of
    // the window nor the mask; the clamp keeps j - q within 32 bits
    const int64_t far = static_cast<int64_t>(kBiasMaxKeys) + 2 * kBiasMaxDistance;
    q = q > far ? far : (q < -kBiasMaxKeys ? -kBiasMaxKeys : q);
    o.r0 = static_cast<int>(-q);
    int64_t n = p.k_len;
    if (p.kv_len) n = min(n, static_cast<int64_t>(p.kv_len[b]));
    if (p.causal) n = min(n, q + 1);
    o.n = static_cast<int>(n < 0 ? 0 : n);
    return o;
}

// The head's biases over the window, and the constants on its two sides.
template <typename T, int EPV>
__device__ __forceinline__ void bias_load_window(const BiasParams& p, const BiasWindow& w, int head,
                                                 float* win, float* low, float* high) {
    auto at = [&](int bucket) {
        const char* t = static_cast<const char*>(p.table);
        const int64_t e = static_cast<int64_t>(bucket) * p.heads + head;
        return get<T, sizeof(T)>(ld_ro<sizeof(T)>(t + e * static_cast<int>(sizeof(T))), 0);
    };
    const int size = w.lo + w.hi + 2 * EPV;
    for (int i = threadIdx.x; i < size; i += blockDim.x)
        win[bias_slot<EPV>(i)] = at(bias_bucket(p, i - w.lo - EPV));
    *low = at(p.half - 1);
    *high = at(p.both ? 2 * p.half - 1 : 0);
}

// Biases of the EPV keys from relative position r on.
template <int EPV>
__device__ __forceinline__ void bias_of(const BiasWindow& w, const float* win, float low, float high,
                                        int r, float (&b)[EPV]) {
    if (r + EPV - 1 <= -w.lo || r >= w.hi) {
        const float c = r >= w.hi ? high : low;
#pragma unroll
        for (int k = 0; k < EPV; ++k) b[k] = c;
    } else {
        const int idx = r + w.lo + EPV;
#pragma unroll
        for (int k = 0; k < EPV; ++k) b[k] = win[bias_slot<EPV>(idx + k)];
    }
}

// Add ds of the EPV keys from relative position r on to the window's sums or
// to the thread's sums of the sides.
template <int EPV>
__device__ __forceinline__ void bias_add(const BiasWindow& w, float* win, float& low, float& high,
                                         int r, const float (&ds)[EPV]) {
    if (r + EPV - 1 <= -w.lo || r >= w.hi) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < EPV; ++k) s += ds[k];
        if (r >= w.hi) high += s; else low += s;
    } else {
        const int idx = r + w.lo + EPV;
#pragma unroll
        for (int k = 0; k < EPV; ++k) win[bias_slot<EPV>(idx + k)] += ds[k];
    }
}

// Fold the windows of `groups` row groups (stride `slots`) and the threads'
// side sums into sums[bucket], and clear them.  All threads of the block.
template <int EPV>
__device__ __forceinline__ void bias_fold(const BiasParams& p, const BiasWindow& w, float* win,
                                          int groups, int slots, float& low, float& high,
                                          double* sums, float2* red) {
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarp = blockDim.x >> 5;
    for (int k = warp; k < p.num_buckets; k += nwarp) {
        const int e = k < p.half ? k : k - p.half;
        const int first = p.edges[e];                        // distances of the bucket
        const int last = e + 1 < p.half ? p.edges[e + 1] - 1 : w.lo + EPV;
        int ra, rb;                                          // relative positions [ra, rb]
        if (k < p.half) {
            ra = -last;
            rb = e == 0 && !p.both ? EPV - 1 : -first;       // one direction: r > 0 is bucket 0
        } else {
            ra = first > 1 ? first : 1;
            rb = e + 1 < p.half ? last : w.hi + EPV - 1;
        }
        float s = 0.f;
        for (int r = ra + lane; r <= rb; r += 32) {
            const int slot = bias_slot<EPV>(r + w.lo + EPV);
            for (int g = 0; g < groups; ++g) {
                s += win[g * slots + slot];
                win[g * slots + slot] = 0.f;
            }
        }
        s = warp_allreduce_sum(s);
        if (lane == 0) sums[k] += static_cast<double>(s);
    }
    const float2 side = block_sum2(low, high, red);          // a barrier: sums[] are written
    if (threadIdx.x == 0) {
        sums[p.half - 1] += static_cast<double>(side.x);
        sums[p.both ? 2 * p.half - 1 : 0] += static_cast<double>(side.y);
    }
    low = high = 0.f;
    __syncthreads();
}

// ------------------------------------------------------- rows of any width --

constexpr int kBiasWideThreads = 256;

// The row is read twice (the second read normally from L2): a running maximum
// and sum, then the outputs.
template <typename T, int VB>
__global__ void __launch_bounds__(kBiasWideThreads) relbias_fwd_wide_kernel(const BiasParams p) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    extern __shared__ float win[];
    __shared__ float2 red[2][kBiasWideThreads / 32];
    pdl_trigger();
    const BiasWindow w(p);
    const int head = blockIdx.x / p.parts;
    const int tid = threadIdx.x;
    pdl_wait();
    float low, high;
    bias_load_window<T, EPV>(p, w, head, win, &low, &high);
    __syncthreads();
    int it = 0;
    for (int row = blockIdx.x - head * p.parts; row < p.head_rows; row += p.parts, ++it) {
        const BiasRow ri = bias_row(p, head, row);
        const char* src = static_cast<const char*>(p.x) + ri.at * static_cast<int>(sizeof(T));
        char* dst = static_cast<char*>(p.out) + ri.at * static_cast<int>(sizeof(T));
        auto load = [&](int i, float (&v)[EPV]) {
            const Vec<VB> x = ld_plain<VB>(src + static_cast<int64_t>(i) * VB);
            float b[EPV];
            bias_of<EPV>(w, win, low, high, ri.r0 + i * EPV, b);
#pragma unroll
            for (int k = 0; k < EPV; ++k)
                v[k] = i * EPV + k < ri.n ? fmaf(get<T, VB>(x, k), p.scale, b[k]) : -INFINITY;
        };
        float m = -INFINITY, s = 0.f;
        for (int i = tid; i < p.nvec && i * EPV < ri.n; i += kBiasWideThreads) {
            float v[EPV];
            load(i, v);
            float mv = m;
#pragma unroll
            for (int k = 0; k < EPV; ++k) mv = fmaxf(mv, v[k]);
            if (mv > m) {
                s *= exp2f((m - mv) * kLog2e);
                m = mv;
            }
            // nothing but -inf so far: -inf adds 0, a NaN is kept
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int k = 0; k < EPV; ++k)
                if (i * EPV + k < ri.n) s += exp2f((v[k] - ref) * kLog2e);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const float mo = __shfl_xor_sync(0xffffffffu, m, d);
            const float so = __shfl_xor_sync(0xffffffffu, s, d);
            pair_fold(m, s, mo, so);
        }
        float2* slot = red[it & 1];
        if ((tid & 31) == 0) slot[tid >> 5] = make_float2(m, s);
        __syncthreads();
        m = -INFINITY;
        s = 0.f;
        for (int k = 0; k < kBiasWideThreads / 32; ++k) pair_fold(m, s, slot[k].x, slot[k].y);
        const float inv = 1.f / s;
        for (int i = tid; i < p.nvec; i += kBiasWideThreads) {
            float o[EPV];
            if (i * EPV < ri.n) {
                float v[EPV];
                load(i, v);
#pragma unroll
                for (int k = 0; k < EPV; ++k)
                    o[k] = i * EPV + k < ri.n ? exp2f((v[k] - m) * kLog2e) * inv : 0.f;
            } else {
#pragma unroll
                for (int k = 0; k < EPV; ++k) o[k] = 0.f;
            }
            st_stream<VB>(dst + static_cast<int64_t>(i) * VB, pack<T, VB>(o));
        }
    }
}

// Two reads of y and dy: the row's dot product, then dx and the sums of ds.
template <typename T, int VB>
__global__ void __launch_bounds__(kBiasWideThreads) relbias_bwd_wide_kernel(const BiasParams p) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    extern __shared__ float win[];
    __shared__ double sums[kBiasMaxBuckets];
    __shared__ float2 red[2][32];
    pdl_trigger();
    const BiasWindow w(p);
    const int head = blockIdx.x / p.parts;
    const int part = blockIdx.x - head * p.parts;
    const int tid = threadIdx.x;
    const int slots = bias_window_slots(w.lo, w.hi, EPV);
    if (p.part) {
        for (int i = tid; i < slots; i += kBiasWideThreads) win[i] = 0.f;
        for (int k = tid; k < p.num_buckets; k += kBiasWideThreads) sums[k] = 0.0;
    }
    __syncthreads();
    pdl_wait();
    float low = 0.f, high = 0.f;
    int it = 0;
    for (int row = part; row < p.head_rows; row += p.parts, ++it) {
        const BiasRow ri = bias_row(p, head, row);
        const int64_t at = ri.at * static_cast<int>(sizeof(T));
        const char* ys = static_cast<const char*>(p.y) + at;
        const char* ds = static_cast<const char*>(p.x) + at;
        char* dst = static_cast<char*>(p.out) + at;
        float dot = 0.f;
        for (int i = tid; i < p.nvec && i * EPV < ri.n; i += kBiasWideThreads) {
            const Vec<VB> yv = ld_plain<VB>(ys + static_cast<int64_t>(i) * VB);
            const Vec<VB> dv = ld_plain<VB>(ds + static_cast<int64_t>(i) * VB);
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < EPV; ++k)
                if (i * EPV + k < ri.n) s = fmaf(get<T, VB>(yv, k), get<T, VB>(dv, k), s);
            dot += s;
        }
        dot = block_sum2(dot, 0.f, red[it & 1]).x;
        for (int i = tid; i < p.nvec; i += kBiasWideThreads) {
            float o[EPV], g[EPV];
#pragma unroll
            for (int k = 0; k < EPV; ++k) o[k] = g[k] = 0.f;
            if (i * EPV < ri.n) {
                const Vec<VB> yv = ld_plain<VB>(ys + static_cast<int64_t>(i) * VB);
                const Vec<VB> dv = ld_plain<VB>(ds + static_cast<int64_t>(i) * VB);
#pragma unroll
                for (int k = 0; k < EPV; ++k) {
                    if (i * EPV + k < ri.n) {
                        g[k] = get<T, VB>(yv, k) * (get<T, VB>(dv, k) - dot);
                        o[k] = g[k] * p.scale;
                    }
                }
                if (p.part) bias_add<EPV>(w, win, low, high, ri.r0 + i * EPV, g);
            }
            st_stream<VB>(dst + static_cast<int64_t>(i) * VB, pack<T, VB>(o));
        }
        if (p.part && it % kBiasFoldRows == kBiasFoldRows - 1)
            bias_fold<EPV>(p, w, win, 1, slots, low, high, sums, red[0]);
    }
    if (p.part) {
        bias_fold<EPV>(p, w, win, 1, slots, low, high, sums, red[0]);
        double* out = p.part + static_cast<int64_t>(blockIdx.x) * p.num_buckets;
        for (int k = tid; k < p.num_buckets; k += kBiasWideThreads) out[k] = sums[k];
    }
}

// dt[k, h] from the CTAs' sums: one CTA per head, a warp per bucket.
constexpr int kBiasReduceThreads = 256;

static __global__ void __launch_bounds__(kBiasReduceThreads)
relbias_reduce_kernel(const BiasParams p) {
    pdl_trigger();
    pdl_wait();
    const int head = blockIdx.x, lane = threadIdx.x & 31;
    for (int k = threadIdx.x >> 5; k < p.num_buckets; k += kBiasReduceThreads / 32) {
        const double* src = p.part + static_cast<int64_t>(head) * p.parts * p.num_buckets + k;
        double s = 0.0;
        for (int c = lane; c < p.parts; c += 32) s += src[static_cast<int64_t>(c) * p.num_buckets];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (lane == 0) p.dtable[static_cast<int64_t>(k) * p.heads + head] = static_cast<float>(s);
    }
}

}  // namespace rmsnorm
