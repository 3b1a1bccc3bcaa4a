// k_relbias.cuh -- row softmax of attention scores with a learned relative
// position bias, and its backward pass.
//
// Scores x[b, h, i, j] (batch, head, query, key).  The query stands at
// q = q_offset + q_start[b] + i, so the key's relative position is r = j - q:
//     v = scale * x + t[bucket(r), h]      over the valid keys of the row,
//     y = exp(v - max v) / sum exp(v - max v),  0 at the other keys.
// Both masks, j < kv_len[b] and (causal) r <= 0, leave a prefix [0, n) of the
// row valid; what is outside it does not matter, and a row with n = 0 is all zero.
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
#include "pairs.cuh"
#include "relbias_launch.h"

namespace rmsnorm {

// Measured (calls back to back, % of the HBM copy peak, bf16 unless fp32 is said):
// forward 256 x 512 x 512 48 us, 82, 128 x 2048 x 2048 356 us, 89, causal (half as many
// bytes read) 354 us, 67, fp32 128 x 2048 x 2048 648 us, 98; backward 128 x 2048 x
// 2048 507 us, 94, causal 429 us, 74, 256 x 512 x 512 77 us, 77, fp32 128 x 2048 x 2048
// 948 us, 100.  Rows of 128 / 32 / 8 keys: forward 87 / 72 / 33, backward 85 / 53 / 28.
// A row costs the same instructions and the same wait for its sum whether its
// mask leaves all or half of it, so masked rows stay further from the bandwidth:
// forward the issue slots (64-68% busy), backward the wait for y and dy (the
// registers of a second row in flight would cost as many resident warps).
// Odd rows: forward fp32 (21, 25, 422, 517) 196 us, 69, backward bf16 (5, 28, 873,
// 761) 125 us, 66.
constexpr int kBiasFoldRows = 64;
constexpr int kBiasFoldTurns = 256;      // the same where rows share a window in turn

template <int EPV>
__device__ __forceinline__ int bias_slot(int idx) {
    return EPV > 1 ? idx + idx / EPV : idx;      // EPV is a power of two
}

// Buckets of one direction: the last one whose edge is at most n.
__device__ __forceinline__ int bias_bucket_of(const BiasParams& p, const int* edges, int n) {
    int lo = 0, hi = p.half;                     // edges[lo] <= n < edges[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (edges[mid] <= n) lo = mid; else hi = mid;
    }
    return lo;
}

// `edges`: p.edges, or a copy in shared memory, which threads of different
// positions read faster than the parameters.
__device__ __forceinline__ int bias_bucket(const BiasParams& p, const int* edges, int r) {
    if (p.both) return bias_bucket_of(p, edges, r < 0 ? -r : r) + (r > 0 ? p.half : 0);
    return bias_bucket_of(p, edges, r < 0 ? -r : 0);
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

__device__ __forceinline__ BiasRow bias_row_of(const BiasParams& p, int head, int b, int i) {
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

__device__ __forceinline__ BiasRow bias_row(const BiasParams& p, int head, int row) {
    const int b = row / p.q_len;
    return bias_row_of(p, head, b, row - b * p.q_len);
}

// The relative positions [ra, rb] of a bucket, the sides' buckets as far as
// -low and high.
__device__ __forceinline__ void bias_bucket_range(const BiasParams& p, int k, int low, int high,
                                                  int* ra, int* rb) {
    const int e = k < p.half ? k : k - p.half;
    const int first = p.edges[e];                            // distances of the bucket
    const bool outer = e + 1 == p.half;
    if (k < p.half) {
        *ra = outer ? -low : 1 - p.edges[e + 1];
        *rb = e == 0 && !p.both ? high : -first;             // one direction: r > 0 is bucket 0
    } else {
        *ra = first > 1 ? first : 1;
        *rb = outer ? high : p.edges[e + 1] - 1;
    }
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
        win[bias_slot<EPV>(i)] = at(bias_bucket(p, p.edges, i - w.lo - EPV));
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

// Fold the window and the threads' side sums into sums[bucket], and clear them.
// All threads of the block.
template <int EPV>
__device__ __forceinline__ void bias_fold(const BiasParams& p, const BiasWindow& w, float* win,
                                          float& low, float& high, double* sums, float2* red) {
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarp = blockDim.x >> 5;
    for (int k = warp; k < p.num_buckets; k += nwarp) {
        int ra, rb;                                          // relative positions [ra, rb]
        bias_bucket_range(p, k, w.lo + EPV, w.hi + EPV - 1, &ra, &rb);
        float s = 0.f;
        for (int r = ra + lane; r <= rb; r += 32) {
            const int slot = bias_slot<EPV>(r + w.lo + EPV);
            s += win[slot];
            win[slot] = 0.f;
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

// A CTA per row, which reads the row's valid keys twice (forward: maximum and sum,
// then the outputs; backward: the dot product, then dx and the sums), at any
// width and alignment; the second read comes from L2.  The wait for the row's
// first pass between the two bounds it: fp32 rows of 20000, 33 and 37% of the HBM
// copy peak.
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
            bias_fold<EPV>(p, w, win, low, high, sums, red[0]);
    }
    if (p.part) {
        bias_fold<EPV>(p, w, win, low, high, sums, red[0]);
        double* out = p.part + static_cast<int64_t>(blockIdx.x) * p.num_buckets;
        for (int k = tid; k < p.num_buckets; k += kBiasWideThreads) out[k] = sums[k];
    }
}

// ------------------------------------------------------ rows in registers --
// G threads per row (p.group: a multiple of 32, or a power of two below 32 for
// several rows per warp), NV vectors per thread, read once.  One exchange per
// row: a warp (lane group) forms its exponentials relative to its own maximum,
// and the (maximum, sum) pairs of a row's warps meet behind one barrier.
//
// exp(v - m) is 2^((v - m) * log2(e)) with the subtraction first: v - m is
// never positive and exact for every key that counts, so scores of any
// magnitude, the type's lowest value included, come out right (an all-lowest
// row is uniform), which folding log2(e) into the scale would overflow.
//
// The window is laid out for whole vectors: vector v of a row starts at window
// position base + EPV * v, so all its vectors have the row's phase base % 4,
// and four copies of the window, each shifted by one position, let every one
// be read (backward: updated) by 16-byte accesses, two for 8 keys, whose even
// and odd chunks lie in separate halves so that neighbouring lanes hit
// neighbouring chunks.  It is padded by two vectors of each side's constant:
// a vector beyond is moved to the padding, so lookups need no bounds.

//
// Accesses are 16-byte vectors whatever the rows' length: with SHIFT (rows that
// are not a multiple of 16 bytes) a row's vector 0 is the one that holds its
// first key, `shift` elements into it, so keys have indices from `shift` on;
// the vectors at its two ends are stored element by element.

// Registers per thread: few enough for resident warps (the row's loads are the only
// ones in flight), at the price of small spills: backward bf16 with 4 vectors 36 to
// 44 bytes a thread, with 6 16, forward bf16 shifted rows 28; fp32 none or 4.
// Measured (% of the HBM copy peak, 4 vectors): bf16 forward 96 / 112 / 128 registers
// 89 / 90 / 90 on rows of 2048 and 41 / 38 / 38 on a decoding step; backward 64 / 72 /
// 80 registers, bf16 rows of 2048 90 / 94 / 96, causal 73 / 75 / 71, of 512 68 / 80 /
// 69, fp32 rows of 1024 89 / 91 / 91.
template <typename T, int NV>
constexpr int bias_fwd_regs() {
    return NV == 4 ? (sizeof(T) == 2 ? 96 : 80) : (sizeof(T) == 2 ? 128 : 104);
}
template <int NV>
constexpr int bias_bwd_regs() { return NV == 4 ? 72 : 96; }

// Where the pair (m, .) stands relative to the maximum M >= m; 1 if both are -inf.
__device__ __forceinline__ float bias_factor(float m, float M) {
    return m == M ? 1.f : exp2f((m - M) * kLog2e);
}

template <int EPV>
struct VecWindow {
    static_assert(EPV == 4 || EPV == 8, "vectors of 16 bytes");
    BiasVecWindow s;
    int lo, hi;
    __device__ __forceinline__ explicit VecWindow(const BiasWindow& w)
        : s(bias_vec_window(w.lo, w.hi, EPV)), lo(w.lo), hi(w.hi) {}
    __device__ __forceinline__ int floats() const { return s.copies * s.copy; }
    // position of relative position r, and the r of position 0
    __device__ __forceinline__ int first() const { return -lo - 2 * EPV; }
    static constexpr int C = 4;                       // copies, and floats of a chunk
    // where copy c keeps position idx >= c
    __device__ __forceinline__ int slot(int c, int idx) const {
        const int d = idx - c, q = d / C, h = d % C;      // C is a power of two, d >= 0
        const int chunk = EPV == 8 ? (q & 1) * s.half + (q >> 1) : q;
        return c * s.copy + chunk * C + h;
    }
};

// A row's view of a window: vector v's chunks are at p0 + v (and p1 + v), v
// moved into [vmin, vmax]; vectors up to vmin are all low, from vmax on all high.
template <int EPV>
struct WindowRow {
    static constexpr int C = VecWindow<EPV>::C;
    int p0, p1;                                       // float offsets
    int vmin, vmax;
    __device__ __forceinline__ WindowRow(const VecWindow<EPV>& w, int r0) {
        const int base = r0 - w.first();              // position of the row's vector 0
        constexpr int SH = EPV == 8 ? 3 : 2;
        const int phase = base & (EPV - 1);           // 0 .. EPV - 1
        const int v0 = base >> SH;                    // whole vectors before it
        vmin = -v0;
        vmax = ((w.lo + w.hi + 3 * EPV - 1 - phase) >> SH) - v0;
        const int c = phase & (C - 1);
        if constexpr (EPV == 8) {
            const int odd = phase >> 2;
            const int a = c * w.s.copy + v0 * C;
            p0 = odd ? a + w.s.half * C : a;
            p1 = odd ? a + C : a + w.s.half * C;
        } else {
            p0 = c * w.s.copy + v0 * C;
            p1 = 0;
        }
    }
    __device__ __forceinline__ int moved(int v) const { return min(max(v, vmin), vmax); }
    __device__ __forceinline__ void read(const float* win, int v, float (&b)[EPV]) const {
        const float4 x = *reinterpret_cast<const float4*>(win + p0 + v * C);
        b[0] = x.x; b[1] = x.y; b[2] = x.z; b[3] = x.w;
        if constexpr (EPV == 8) {
            const float4 y = *reinterpret_cast<const float4*>(win + p1 + v * C);
            b[4] = y.x; b[5] = y.y; b[6] = y.z; b[7] = y.w;
        }
    }
    __device__ __forceinline__ void write(float* win, int v, const float (&b)[EPV]) const {
        *reinterpret_cast<float4*>(win + p0 + v * C) = make_float4(b[0], b[1], b[2], b[3]);
        if constexpr (EPV == 8)
            *reinterpret_cast<float4*>(win + p1 + v * C) = make_float4(b[4], b[5], b[6], b[7]);
    }
};

// The rows of one group of a CTA, first + k * step of its head, without a
// division per row.  Rows behind the head's last one have no valid keys and
// are not written (at < 0).
struct BiasRows {
    int row, b, i;
    int step, step_b, step_i;
    __device__ __forceinline__ BiasRows(const BiasParams& p, int first, int step_)
        : row(first), b(first / p.q_len), i(first - b * p.q_len), step(step_),
          step_b(step_ / p.q_len), step_i(step_ - step_b * p.q_len) {}
    __device__ __forceinline__ BiasRow get(const BiasParams& p, int head) const {
        BiasRow o;
        o.at = -1;
        o.n = o.r0 = 0;
        if (row < p.head_rows) o = bias_row_of(p, head, b, i);
        return o;
    }
    __device__ __forceinline__ void next(const BiasParams& p) {
        row += step;
        b += step_b;
        i += step_i;
        if (i >= p.q_len) {
            i -= p.q_len;
            ++b;
        }
    }
};

// What the warp has of vector number i of its threads, one bit each: valid keys
// only (full), none at all, or (neither) some; valid keys are [from, to).  A
// masked row then pays the per-element masks only where its valid keys end.
template <int EPV, int NV>
struct VecClasses {
    uint32_t f = 0, s = 0;
    __device__ __forceinline__ VecClasses(int from, int to, int t, int G) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = (i * G + t) * EPV;
            f |= __all_sync(0xffffffffu, j >= from && j + EPV <= to) ? 1u << i : 0u;
            s |= __any_sync(0xffffffffu, j < to) ? 1u << i : 0u;
        }
    }
    __device__ __forceinline__ bool all() const { return f == (1u << NV) - 1; }
    __device__ __forceinline__ bool full(int i) const { return f >> i & 1u; }
    __device__ __forceinline__ bool none(int i) const { return !(s >> i & 1u); }
};

// A row in vectors: element `at` (a multiple of EPV) is its vector 0's first,
// its keys have indices [shift, shift + k_len), the valid ones [shift, to).
template <bool SHIFT, int EPV>
struct VecRow {
    int64_t at;
    int shift, to, end;
    bool here, cut;               // cut: its last valid keys' vector passes the array's end
    __device__ __forceinline__ VecRow(const BiasRow& r, int k_len, int64_t total) {
        shift = SHIFT ? static_cast<int>(r.at & (EPV - 1)) : 0;
        at = r.at - shift;
        to = r.n > 0 ? r.n + shift : 0;
        end = k_len + shift;
        here = r.at >= 0;
        cut = SHIFT && at + (to + EPV - 1) / EPV * EPV > total;
    }
};

// Vector at element e of an array; `cut`: only what of it lies inside the
// array of `total` elements.
template <typename T>
__device__ __forceinline__ Vec<16> ld_vec(const void* base, int64_t e, bool cut, int64_t total) {
    constexpr int EPV = VecTraits<T, 16>::kElems;
    const char* p = static_cast<const char*>(base) + e * static_cast<int>(sizeof(T));
    if (!cut) return ld_stream<16>(p);
    Vec<16> v = zero_vec();
#pragma unroll
    for (int k = 0; k < EPV; ++k) {
        if (e + k < total) {
            if constexpr (sizeof(T) == 4) {
                v.u[k] = ld_stream<4>(p + 4 * k).u[0];
            } else {
                v.u[k / 2] |= static_cast<uint32_t>(ld_stream<2>(p + 2 * k).h) << (16 * (k & 1));
            }
        }
    }
    return v;
}

// Store a row's vector j / EPV: whole, or the elements inside the row.
// `first`: it may be the row's first one.
template <typename T, bool SHIFT, class Row>
__device__ __forceinline__ void st_vec(void* base, const Row& r, bool first, int j,
                                       const Vec<16>& v) {
    constexpr int EPV = VecTraits<T, 16>::kElems;
    char* p = static_cast<char*>(base) + (r.at + j) * static_cast<int>(sizeof(T));
    if (!SHIFT || ((!first || j >= r.shift) && j + EPV <= r.end)) {
        st_stream<16>(p, v);
        return;
    }
#pragma unroll
    for (int k = 0; k < EPV; ++k) {
        if ((!first || j + k >= r.shift) && j + k < r.end) {
            if constexpr (sizeof(T) == 4) {
                Vec<4> o;
                o.u[0] = v.u[k];
                st_stream<4>(p + 4 * k, o);
            } else {
                Vec<2> o;
                o.h = static_cast<uint16_t>(v.u[k / 2] >> (16 * (k & 1)));
                st_stream<2>(p + 2 * k, o);
            }
        }
    }
}

template <typename T, int NV, bool SHIFT>
__global__ void __maxnreg__((bias_fwd_regs<T, NV>())) relbias_fwd_rowreg_kernel(const BiasParams p) {
    constexpr int EPV = VecTraits<T, 16>::kElems;
    constexpr int PN = kPairs<T>;
    using L = Lanes;
    extern __shared__ __align__(16) float win[];
    __shared__ float2 red[2][32];
    __shared__ float biases[kBiasMaxBuckets];
    __shared__ int edges[kBiasMaxBuckets];
    pdl_trigger();
    const BiasWindow bw(p);
    const VecWindow<EPV> w(bw);
    const int G = p.group;
    const int width = G < 32 ? G : 32;
    const int tid = threadIdx.x;
    const int g = tid / G;
    const int t = tid - g * G;
    const int warp = tid >> 5, lane = tid & 31;
    const int wpg = G >> 5;
    const int gw0 = g * wpg;
    const int rpc = p.rows_per_cta;
    const int head = blockIdx.x / p.parts;
    int merge_width = 1;
    while (merge_width < wpg) merge_width <<= 1;
    int block = blockIdx.x - head * p.parts;
    const int nblocks = (p.head_rows + rpc - 1) / rpc;
    BiasRows rows(p, block * rpc + g, p.parts * rpc);
    pdl_wait();

    using Row = VecRow<SHIFT, EPV>;
    Vec<16> cur[NV], nxt[NV];
    auto load = [&](Vec<16> (&dst)[NV], const Row& r) {
        auto vectors = [&](auto cut) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = (i * G + t) * EPV;
                if (j < r.to) dst[i] = ld_vec<T>(p.x, r.at + j, cut && j + EPV > r.to, p.elems);
            }
        };
        if (r.cut) vectors(std::true_type()); else vectors(std::false_type());
    };
    BiasRow info = rows.get(p, head);
    Row ri(info, p.k_len, p.elems);
    int r0 = info.r0 - ri.shift;                 // relative position of index 0
    load(cur, ri);
    for (int k = tid; k < p.num_buckets; k += blockDim.x) {
        const char* table = static_cast<const char*>(p.table);
        const int64_t e = static_cast<int64_t>(k) * p.heads + head;
        biases[k] = get<T, sizeof(T)>(ld_ro<sizeof(T)>(table + e * static_cast<int>(sizeof(T))), 0);
        edges[k] = p.edges[k];
    }
    __syncthreads();
    for (int idx = tid; idx < w.s.size; idx += blockDim.x) {
        const float v = biases[bias_bucket(p, edges, w.first() + idx)];
        for (int c = 0; c < w.C && c <= idx; ++c) win[w.slot(c, idx)] = v;
    }
    __syncthreads();
    const L scale = L::all(p.scale), log2e = L::all(kLog2e);
    for (int it = 0; block < nblocks; block += p.parts, ++it) {
        rows.next(p);
        info = rows.get(p, head);
        const Row rn(info, p.k_len, p.elems);
        load(nxt, rn);
        L e[NV * PN];
        float m = -INFINITY, s = 0.f;
        const WindowRow<EPV> wr(w, r0);
        const VecClasses<EPV, NV> is(ri.shift, ri.to, t, G);
        // each pass twice: `all` vectors of the warp valid in full, or by class
        auto scores = [&](auto all) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!all && is.none(i)) continue;
                const int v = i * G + t, j = v * EPV;
                // a lookup for every vector: asking first whether the whole warp's are
                // outside the window costs more (fp32 rows of 517 217 / 203 us, bf16 of
                // 520 87 / 64)
                float b[EPV];
                wr.read(win, wr.moved(v), b);
#pragma unroll
                for (int k = 0; k < PN; ++k)
                    e[i * PN + k] = fma(lanes<T>(cur[i], k), scale, L::of(b + 2 * k));
                if (!all && !is.full(i)) {           // masked keys
#pragma unroll
                    for (int k = 0; k < PN; ++k) {
                        float a[2];
                        e[i * PN + k].put(a);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int at = j + 2 * k + h;
                            if (at >= ri.to || (SHIFT && i == 0 && at < ri.shift)) a[h] = -INFINITY;
                        }
                        e[i * PN + k] = L::of(a);
                    }
                }
#pragma unroll
                for (int k = 0; k < PN; ++k) m = e[i * PN + k].largest(m);
            }
        };
        const bool all = is.all();
        if (all) scores(std::true_type()); else scores(std::false_type());
        m = width == 32 ? warp_allreduce_max(m) : group_allreduce_max(m, width);
        const L minus = L::all(m == -INFINITY ? 0.f : -m);
        L s0 = L::all(0.f), s1 = L::all(0.f);
        auto exponentials = [&](auto all) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!all && is.none(i)) continue;
#pragma unroll
                for (int k = 0; k < PN; ++k) {
                    float a[2];
                    ((e[i * PN + k] + minus) * log2e).put(a);
#pragma unroll
                    for (int h = 0; h < 2; ++h) a[h] = row_exp_arg<T>(a[h]);
                    e[i * PN + k] = L::of(a);
                    if (k & 1) s1 = s1 + e[i * PN + k]; else s0 = s0 + e[i * PN + k];
                }
            }
        };
        if (all) exponentials(std::true_type()); else exponentials(std::false_type());
        s = share_sum((s0 + s1).total(), width);
        float f = 1.f;
        if (wpg > 1) {
            float2* slot = red[it & 1];
            if (lane == 0) slot[warp] = make_float2(m, s);
            __syncthreads();
            float2 o = make_float2(-INFINITY, 0.f);
            if (lane < wpg) o = slot[gw0 + lane];
            const float M = __shfl_sync(0xffffffffu, group_allreduce_max(o.x, merge_width), 0);
            s = group_allreduce_sum(o.y * bias_factor(o.x, M), merge_width);
            s = __shfl_sync(0xffffffffu, s, 0);
            f = bias_factor(m, M);
        }
        // a row of -inf: s = 0, 0 * (1 / 0) = NaN at its valid keys
        const L inv = L::all(f / s);
        auto outputs = [&](auto all) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = (i * G + t) * EPV;
                if (!all && is.none(i)) {
                    if (ri.here && j < ri.end) st_vec<T, SHIFT>(p.out, ri, i == 0, j, zero_vec());
                    continue;
                }
                float o[EPV];
#pragma unroll
                for (int k = 0; k < PN; ++k) (e[i * PN + k] * inv).put(o + 2 * k);
                if (all || is.full(i)) {
                    st_vec<T, false>(p.out, ri, false, j, pack<T, 16>(o));
                } else if (ri.here && j < ri.end) {
#pragma unroll
                    for (int k = 0; k < EPV; ++k)
                        if (j + k >= ri.to) o[k] = 0.f;
                    st_vec<T, SHIFT>(p.out, ri, i == 0, j, pack<T, 16>(o));
                }
            }
        };
        if (all) outputs(std::true_type()); else outputs(std::false_type());
        ri = rn;
        r0 = info.r0 - rn.shift;
#pragma unroll
        for (int i = 0; i < NV; ++i) cur[i] = nxt[i];
    }
}

// Fold the windows of `groups` row groups and the threads' side sums into
// sums[bucket], and clear them: first a thread per position over all groups and
// copies (into `total`, w.s.size floats), then a warp per bucket.  All threads
// of the block.
template <int EPV>
__device__ __forceinline__ void bias_fold_vec(const BiasParams& p, const VecWindow<EPV>& w,
                                              float* wins, float* total, int groups, float& low,
                                              float& high, double* sums, float2* red) {
    constexpr int C = VecWindow<EPV>::C;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarp = blockDim.x >> 5;
    for (int idx = threadIdx.x; idx < w.s.size; idx += blockDim.x) {
        float s[C];
#pragma unroll
        for (int c = 0; c < C; ++c) s[c] = 0.f;
        for (int g = 0; g < groups; ++g) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (c <= idx) {
                    float* at = wins + g * w.floats() + w.slot(c, idx);
                    s[c] += *at;
                    *at = 0.f;
                }
            }
        }
#pragma unroll
        for (int c = 1; c < C; ++c) s[0] += s[c];
        total[idx] = s[0];
    }
    const float2 side = block_sum2(low, high, red);          // a barrier: total[] is written
    for (int k = warp; k < p.num_buckets; k += nwarp) {
        int ra, rb;                                          // relative positions [ra, rb]
        bias_bucket_range(p, k, w.lo + 2 * EPV, w.hi + 2 * EPV - 1, &ra, &rb);
        float s = 0.f;
        for (int r = ra + lane; r <= rb; r += 32) s += total[r - w.first()];
        s = warp_allreduce_sum(s);
        if (lane == 0) {
            double d = static_cast<double>(s);
            if (k == p.half - 1) d += static_cast<double>(side.x);
            if (k == (p.both ? 2 * p.half - 1 : 0)) d += static_cast<double>(side.y);
            sums[k] += d;
        }
    }
    low = high = 0.f;
    __syncthreads();
}

// Backward: y and dy of a row in registers, the row's dot product exchanged
// behind one barrier, which also orders the rows' updates of the group's
// window (rows_per_cta windows per CTA).  TURNS, several rows to a warp: p.turns
// neighbouring groups share a window and add to it one after the other, vector by
// vector, with the warp in step: windows no longer decide how many warps an SM
// holds, and the order of the additions stays fixed.
template <typename T, int NV, bool SHIFT, bool TURNS>
__global__ void __maxnreg__(bias_bwd_regs<NV>()) relbias_bwd_rowreg_kernel(const BiasParams p) {
    constexpr int EPV = VecTraits<T, 16>::kElems;
    constexpr int PN = kPairs<T>;
    using L = Lanes;
    extern __shared__ __align__(16) float wins[];
    __shared__ double sums[kBiasMaxBuckets];
    __shared__ float red[2][32];
    __shared__ float2 fold_red[32];
    pdl_trigger();
    const BiasWindow bw(p);
    const VecWindow<EPV> w(bw);
    const int G = p.group;
    const int width = G < 32 ? G : 32;
    const int tid = threadIdx.x;
    const int g = tid / G;
    const int t = tid - g * G;
    const int warp = tid >> 5, lane = tid & 31;
    const int wpg = G >> 5;
    const int gw0 = g * wpg;
    const int rpc = p.rows_per_cta;
    const int head = blockIdx.x / p.parts;
    int merge_width = 1;
    while (merge_width < wpg) merge_width <<= 1;
    const int turns = TURNS ? p.turns : 1;
    const int windows = TURNS ? rpc / turns : rpc;
    float* win = wins + (TURNS ? g / turns : g) * w.floats();
    float* total = wins + windows * w.floats();
    if (p.part) {
        for (int i = tid; i < windows * w.floats(); i += blockDim.x) wins[i] = 0.f;
        for (int k = tid; k < p.num_buckets; k += blockDim.x) sums[k] = 0.0;
    }
    int block = blockIdx.x - head * p.parts;
    const int nblocks = (p.head_rows + rpc - 1) / rpc;
    BiasRows rows(p, block * rpc + g, p.parts * rpc);
    __syncthreads();
    pdl_wait();

    const L scale = L::all(p.scale);
    const int fold_every = TURNS ? max(1, min(kBiasFoldRows, kBiasFoldTurns / turns)) : kBiasFoldRows;
    float low = 0.f, high = 0.f;
    for (int it = 0; block < nblocks; block += p.parts, ++it, rows.next(p)) {
        const BiasRow info = rows.get(p, head);
        const VecRow<SHIFT, EPV> ri(info, p.k_len, p.elems);
        const WindowRow<EPV> wr(w, info.r0 - ri.shift);
        const VecClasses<EPV, NV> is(ri.shift, ri.to, t, G);
        const bool all = is.all();
        Vec<16> y[NV], d[NV];
        auto load = [&](auto cut) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = (i * G + t) * EPV;
                if (j < ri.to) {
                    y[i] = ld_vec<T>(p.y, ri.at + j, cut && j + EPV > ri.to, p.elems);
                    d[i] = ld_vec<T>(p.x, ri.at + j, cut && j + EPV > ri.to, p.elems);
                }
            }
        };
        if (ri.cut) load(std::true_type()); else load(std::false_type());
        L s0 = L::all(0.f), s1 = L::all(0.f);
        // each pass twice: `all` vectors of the warp valid in full, or by class
        auto products = [&](auto all) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!all && is.none(i)) continue;
                if (!all && !is.full(i)) {           // clear what is not a valid key
                    const int j = (i * G + t) * EPV;
                    clear_from<T>(y[i], max(ri.to - j, 0));
                    clear_from<T>(d[i], max(ri.to - j, 0));
                    if (SHIFT && i == 0) {
                        clear_below<T>(y[i], ri.shift - j);
                        clear_below<T>(d[i], ri.shift - j);
                    }
                }
#pragma unroll
                for (int k = 0; k < PN; ++k) {
                    if (k & 1) s1 = fma(lanes<T>(y[i], k), lanes<T>(d[i], k), s1);
                    else s0 = fma(lanes<T>(y[i], k), lanes<T>(d[i], k), s0);
                }
            }
        };
        if (all) products(std::true_type()); else products(std::false_type());
        float dot = share_sum((s0 + s1).total(), width);
        if (wpg > 1) {
            float* slot = red[it & 1];
            if (lane == 0) slot[warp] = dot;
            __syncthreads();
            dot = group_allreduce_sum(lane < wpg ? slot[gw0 + lane] : 0.f, merge_width);
            dot = __shfl_sync(0xffffffffu, dot, 0);
        } else {
            __syncwarp();
        }
        const L minus = L::all(-dot), zero = L::all(0.f);
        // what was cleared stays 0 in y * (dy - dot) unless the dot product is
        // infinite or NaN
        const bool sound = fabsf(dot) < INFINITY;
        auto outputs = [&](auto all) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = i * G + t, j = v * EPV;
                if (!all && is.none(i)) {
                    if (ri.here && j < ri.end) st_vec<T, SHIFT>(p.out, ri, i == 0, j, zero_vec());
                    continue;
                }
                L gk[PN];
#pragma unroll
                for (int k = 0; k < PN; ++k)
                    gk[k] = lanes<T>(y[i], k) * (lanes<T>(d[i], k) + minus);
                if (!all && !sound && !is.full(i)) {
#pragma unroll
                    for (int k = 0; k < PN; ++k) {
                        float a[2];
                        gk[k].put(a);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int at = j + 2 * k + h;
                            if (at >= ri.to || (SHIFT && i == 0 && at < ri.shift)) a[h] = 0.f;
                        }
                        gk[k] = L::of(a);
                    }
                }
                float o[EPV];
#pragma unroll
                for (int k = 0; k < PN; ++k) fma(gk[k], scale, zero).put(o + 2 * k);   // -0: 0
                if (all || is.full(i)) st_vec<T, false>(p.out, ri, false, j, pack<T, 16>(o));
                else if (ri.here && j < ri.end) st_vec<T, SHIFT>(p.out, ri, i == 0, j, pack<T, 16>(o));
                // to the window, or to the thread's sums of the sides
                auto add = [&](bool to_window) {
                    if (to_window) {
                        float a[EPV];
                        wr.read(win, v, a);
#pragma unroll
                        for (int k = 0; k < PN; ++k) (L::of(a + 2 * k) + gk[k]).put(a + 2 * k);
                        wr.write(win, v, a);
                    } else {
                        L sum = gk[0];
#pragma unroll
                        for (int k = 1; k < PN; ++k) sum = sum + gk[k];
                        if (v >= wr.vmax) high += sum.total(); else low += sum.total();
                    }
                };
                const bool inside = v > wr.vmin && v < wr.vmax;
                if constexpr (TURNS) {
                    const bool mine = all || j < ri.to;
                    if (mine && !inside) add(false);
                    for (int turn = 0; turn < turns; ++turn) {
                        if (mine && inside && (g & (turns - 1)) == turn) add(true);
                        __syncwarp();
                    }
                } else if (p.part && (all || j < ri.to)) {
                    if (inside) add(true); else add(false);
                }
            }
        };
        if (all) outputs(std::true_type()); else outputs(std::false_type());
        if (p.part && it % fold_every == fold_every - 1)
            bias_fold_vec<EPV>(p, w, wins, total, windows, low, high, sums, fold_red);
    }
    if (p.part) {
        bias_fold_vec<EPV>(p, w, wins, total, windows, low, high, sums, fold_red);
        double* to = p.part + static_cast<int64_t>(blockIdx.x) * p.num_buckets;
        for (int k = tid; k < p.num_buckets; k += blockDim.x) to[k] = sums[k];
    }
}

// dt[k, h] from the CTAs' sums: blockIdx.x is the head, a warp per bucket.
constexpr int kBiasReduceThreads = 256;

static __global__ void __launch_bounds__(kBiasReduceThreads)
relbias_reduce_kernel(const BiasParams p) {
    pdl_trigger();
    pdl_wait();
    const int head = blockIdx.x, lane = threadIdx.x & 31;
    const int k = (blockIdx.y * kBiasReduceThreads + threadIdx.x) >> 5;
    if (k >= p.num_buckets) return;
    const double* src = p.part + static_cast<int64_t>(head) * p.parts * p.num_buckets + k;
    double s = 0.0;
#pragma unroll 4
    for (int c = lane; c < p.parts; c += 32) s += src[static_cast<int64_t>(c) * p.num_buckets];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) p.dtable[static_cast<int64_t>(k) * p.heads + head] = static_cast<float>(s);
}

}  // namespace rmsnorm
