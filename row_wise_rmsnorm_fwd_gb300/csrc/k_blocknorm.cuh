// k_blocknorm.cuh -- the boundary between two blocks (formulas in
// include/rmsnorm_block.h): kernels for any width and alignment.
#pragma once
#include "blocknorm_launch.h"
#include "common.cuh"
#include "integers.cuh"

namespace rmsnorm {

constexpr int kBlockRowsThreads = 256;
constexpr int kBlockColsThreads = 128;

// Sums of N values over the block (at most 32 warps); all threads get the same
// bits.  red: N * 32 slots, free again after the caller's next barrier.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* red) {
    const int warp = threadIdx.x >> 5, n = blockDim.x >> 5;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = warp_allreduce_sum(v[k]);
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) red[warp * N + k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = 0.f;
        for (int w = 0; w < n; ++w) v[k] += red[w * N + k];
    }
}

// One vector widened; ones where there are no weights.
template <typename T, int VB>
__device__ __forceinline__ void widen_ro(float (&f)[VecTraits<T, VB>::kElems], const char* from) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    Vec<VB> v;
    if (from) v = ld_ro<VB>(from);
#pragma unroll
    for (int k = 0; k < EPV; ++k) f[k] = from ? get<T, VB>(v, k) : 1.f;
}

__device__ __forceinline__ const char* at_or_null(const void* p, int64_t at) {
    return p ? static_cast<const char*>(p) + at : nullptr;
}

// Forward: a CTA per row, which is read once for each sum and once for the
// outputs (again normally from L2).  Dependent reads with a block barrier
// between them bound it.  A thread reads an element of x and residual for
// the last time right before it writes that element of h and y, so either may
// be written in place.
template <typename T, int VB>
__global__ void __launch_bounds__(kBlockRowsThreads) blocknorm_fwd_any_kernel(const BlockParams p) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    __shared__ float red[2][32];
    pdl_trigger();
    pdl_wait();
    const int64_t row_bytes = static_cast<int64_t>(p.hidden) * sizeof(T);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const char* xs = static_cast<const char*>(p.x) + row * row_bytes;
        const char* rs = static_cast<const char*>(p.residual) + row * row_bytes;
        const char* gate = at_or_null(p.gate, row / p.gate_rows * row_bytes);
        float rx = 1.f;
        if (p.post) {
            float s[1] = {0.f};
            for (int i = threadIdx.x; i < p.nvec; i += kBlockRowsThreads) {
                const Vec<VB> v = ld_plain<VB>(xs + static_cast<int64_t>(i) * VB);
                float t = 0.f;
#pragma unroll
                for (int k = 0; k < EPV; ++k) t = fmaf(get<T, VB>(v, k), get<T, VB>(v, k), t);
                s[0] += t;
            }
            block_sums<1>(s, red[0]);
            rx = rsqrtf(fmaf(s[0], p.inv_hidden, p.post_eps));
        }
        auto stream = [&](int i, float (&h)[EPV]) {
            const int64_t at = static_cast<int64_t>(i) * VB;
            const Vec<VB> xv = ld_plain<VB>(xs + at);
            const Vec<VB> rv = ld_plain<VB>(rs + at);
            float w[EPV], g[EPV];
            widen_ro<T, VB>(w, at_or_null(p.post ? p.post_w : nullptr, at));
            widen_ro<T, VB>(g, gate ? gate + at : nullptr);
#pragma unroll
            for (int k = 0; k < EPV; ++k) {
                const float n = get<T, VB>(xv, k) * rx * w[k];
                h[k] = fmaf(p.residual_scale, get<T, VB>(rv, k), p.branch_scale * (g[k] * n));
            }
        };
        float rh = 0.f;
        if (p.pre) {
            float s[1] = {0.f};
            for (int i = threadIdx.x; i < p.nvec; i += kBlockRowsThreads) {
                float h[EPV], t = 0.f;
                stream(i, h);
#pragma unroll
                for (int k = 0; k < EPV; ++k) t = fmaf(h[k], h[k], t);
                s[0] += t;
            }
            block_sums<1>(s, red[1]);
            rh = rsqrtf(fmaf(s[0], p.inv_hidden, p.pre_eps));
        }
        for (int i = threadIdx.x; i < p.nvec; i += kBlockRowsThreads) {
            const int64_t at = static_cast<int64_t>(i) * VB;
            float h[EPV], y[EPV];
            stream(i, h);
            if (p.pre) {
                float w[EPV];
                widen_ro<T, VB>(w, at_or_null(p.pre_w, at));
#pragma unroll
                for (int k = 0; k < EPV; ++k) y[k] = h[k] * rh * w[k];
            }
            st_stream<VB>(static_cast<char*>(p.h) + row * row_bytes + at, pack<T, VB>(h));
            if (p.pre) st_stream<VB>(static_cast<char*>(p.y) + row * row_bytes + at, pack<T, VB>(y));
        }
        __syncthreads();        // red is free again: with one norm nothing else says so
    }
}

// Forward, rows of vectors of less than 16 bytes that are wide enough for a CTA of their own: as
// above, but the row is held in registers, kBlockRegsVecs vectors to a thread, and read once,
// while the row before it is worked on.  Measured (us, this / the kernel above / staged in
// pieces, k_blocknorm_staged.cuh): fp32 2555 x 2050 19.1 / 24.4 / 27.4 (21.6 without the next
// row under way), 32768 x 2050 183 / 225 / 294, 131072 x 258 138 / 355 / 214,
// 65536 x 1027 258 / 301 / 329, bf16 32768 x 4100 257 / 295 / 332, 65536 x 2050 357 / 424 / 373,
// 131072 x 515 308 / 494 / 387.  Twice as many vectors to a thread: bf16 30000 x 8002 487 / 541 /
// 592 (half as many 583), fp32 16384 x 8190 367 / 536, 16384 x 12002 954 / 898.
// AHEAD: the next row is loaded while one is worked on (with twice as many vectors to a thread
// there are no registers for it).
template <typename T, int VB, int NV, bool AHEAD>
__global__ void __launch_bounds__(kBlockRegsMaxThreads, 1) blocknorm_fwd_regs_kernel(const BlockParams p) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    __shared__ float red[2][2][32];
    pdl_trigger();
    pdl_wait();
    const int64_t row_bytes = static_cast<int64_t>(p.hidden) * sizeof(T);
    const int n = static_cast<int>(blockDim.x);
    const int count = (p.nvec - static_cast<int>(threadIdx.x) + n - 1) / n;      // vectors of this thread
    const int64_t mine = static_cast<int64_t>(threadIdx.x) * VB;
    const int apart = n * VB;
    int it = 0;
    Vec<VB> nx[NV], nr[NV];
    auto load_row = [&](int64_t row, Vec<VB> (&x)[NV], Vec<VB> (&r)[NV]) {
        const char* xs = static_cast<const char*>(p.x) + row * row_bytes + mine;
        const char* rs = static_cast<const char*>(p.residual) + row * row_bytes + mine;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (i < count) {
                x[i] = ld_stream<VB>(xs + i * apart);
                r[i] = ld_stream<VB>(rs + i * apart);
            }
        }
    };
    if constexpr (AHEAD) load_row(blockIdx.x, nx, nr);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, it ^= 1) {
        const char* gate = at_or_null(p.gate, row / p.gate_rows * row_bytes + mine);
        const char* post_w = at_or_null(p.post ? p.post_w : nullptr, mine);
        const char* pre_w = at_or_null(p.pre_w, mine);
        Vec<VB> x[NV], r[NV];
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                x[i] = nx[i];
                r[i] = nr[i];
            }
            if (row + gridDim.x < p.rows) load_row(row + gridDim.x, nx, nr);
        } else {
            load_row(row, x, r);
        }
        float scale = p.branch_scale;
        if (p.post) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i < count) {
#pragma unroll
                    for (int k = 0; k < EPV; ++k) s[0] = fmaf(get<T, VB>(x[i], k), get<T, VB>(x[i], k), s[0]);
                }
            }
            block_sums<1>(s, red[it][0]);
            scale *= rsqrtf(fmaf(s[0], p.inv_hidden, p.post_eps));
        }
        float h[NV][EPV];
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (i < count) {
                float w[EPV], g[EPV];
                widen_ro<T, VB>(w, post_w ? post_w + i * apart : nullptr);
                widen_ro<T, VB>(g, gate ? gate + i * apart : nullptr);
#pragma unroll
                for (int k = 0; k < EPV; ++k) {
                    const float b = get<T, VB>(x[i], k) * scale * (w[k] * g[k]);
                    h[i][k] = fmaf(p.residual_scale, get<T, VB>(r[i], k), b);
                    s[0] = fmaf(h[i][k], h[i][k], s[0]);
                }
                st_stream<VB>(static_cast<char*>(p.h) + row * row_bytes + mine + i * apart, pack<T, VB>(h[i]));
            }
        }
        if (p.pre) {
            block_sums<1>(s, red[it][1]);
            const float rh = rsqrtf(fmaf(s[0], p.inv_hidden, p.pre_eps));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i < count) {
                    float w[EPV];
                    widen_ro<T, VB>(w, pre_w ? pre_w + i * apart : nullptr);
#pragma unroll
                    for (int k = 0; k < EPV; ++k) w[k] = h[i][k] * rh * w[k];
                    st_stream<VB>(static_cast<char*>(p.y) + row * row_bytes + mine + i * apart, pack<T, VB>(w));
                }
            }
        }
    }
}

// ------------------------------------------------------------------ backward --
//
// With u = post_w * gate and q = u * x, D = dh + rh * (g - h * kh), the row's last sum
//     sum f x = branch_scale * (sum q dh + rh * (sum q g - kh * sum q h))
// is linear in what the norm of h puts into D, so all six sums of a row come
// from one pass over it, with one exchange.  Nothing is lost by that: it is off by
// roundings of sum |q g|, as it would be with each D rounded before the sum.
// The factors are kept as kh = (sum(g h) / H * rh) * rh: rh^3 at once would overflow
// for rows whose squares are near fp32's smallest numbers, though D does not.

struct BlockFactors {
    float rh, kh;     // D = dh + rh * (g - h * kh)
    float rx, kx;     // dx = rx * (f - x * kx)
};

// s: sums of h^2, g h, x^2, q dh, q g, q h.
__device__ __forceinline__ BlockFactors block_factors(const float (&s)[6], const BlockParams& p) {
    BlockFactors f{0.f, 0.f, 1.f, 0.f};
    float dot = s[3];
    if (p.pre) {
        f.rh = rsqrtf(fmaf(s[0], p.inv_hidden, p.pre_eps));
        f.kh = (s[1] * p.inv_hidden * f.rh) * f.rh;
        dot = fmaf(f.rh, fmaf(-f.kh, s[5], s[4]), dot);
    }
    if (p.post) {
        f.rx = rsqrtf(fmaf(s[2], p.inv_hidden, p.post_eps));
        f.kx = (p.branch_scale * dot * p.inv_hidden * f.rx) * f.rx;
    }
    return f;
}

// Any width: the factors of each row ...  (Together, us and % of the HBM copy peak: bf16 65536 x
// 8192 2275 (42), fp32 16384 x 4097 773 (31): every array is read twice, with a block barrier
// for each row.)
template <typename T, int VB>
__global__ void __launch_bounds__(kBlockRowsThreads) blocknorm_bwd_rows_kernel(const BlockParams p) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    __shared__ float red[2][6 * 32];
    pdl_trigger();
    pdl_wait();
    const int64_t row_bytes = static_cast<int64_t>(p.hidden) * sizeof(T);
    int it = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, it ^= 1) {
        const char* xs = static_cast<const char*>(p.x) + row * row_bytes;
        const char* ds = at_or_null(p.dh, row * row_bytes);
        const char* ys = at_or_null(p.pre ? p.dy : nullptr, row * row_bytes);
        const char* hs = at_or_null(p.pre ? p.h_in : nullptr, row * row_bytes);
        const char* gate = at_or_null(p.gate, row / p.gate_rows * row_bytes);
        float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int i = threadIdx.x; i < p.nvec; i += kBlockRowsThreads) {
            const int64_t at = static_cast<int64_t>(i) * VB;
            float q[EPV];
            float t[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (p.post) {
                const Vec<VB> xv = ld_plain<VB>(xs + at);
                float w[EPV], gt[EPV];
                widen_ro<T, VB>(w, at_or_null(p.post_w, at));
                widen_ro<T, VB>(gt, gate ? gate + at : nullptr);
#pragma unroll
                for (int k = 0; k < EPV; ++k) {
                    const float x = get<T, VB>(xv, k);
                    q[k] = gt[k] * w[k] * x;
                    t[2] = fmaf(x, x, t[2]);
                }
                if (ds) {
                    const Vec<VB> dv = ld_plain<VB>(ds + at);
#pragma unroll
                    for (int k = 0; k < EPV; ++k) t[3] = fmaf(q[k], get<T, VB>(dv, k), t[3]);
                }
            }
            if (p.pre) {
                const Vec<VB> yv = ld_plain<VB>(ys + at);
                const Vec<VB> hv = ld_plain<VB>(hs + at);
                float w[EPV];
                widen_ro<T, VB>(w, at_or_null(p.pre_w, at));
#pragma unroll
                for (int k = 0; k < EPV; ++k) {
                    const float h = get<T, VB>(hv, k), g = get<T, VB>(yv, k) * w[k];
                    t[0] = fmaf(h, h, t[0]);
                    t[1] = fmaf(g, h, t[1]);
                    if (p.post) {
                        t[4] = fmaf(q[k], g, t[4]);
                        t[5] = fmaf(q[k], h, t[5]);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 6; ++k) s[k] += t[k];
        }
        block_sums<6>(s, red[it]);
        if (threadIdx.x == 0) {
            const BlockFactors f = block_factors(s, p);
            p.row_stats[row] = make_float4(f.rh, f.kh, f.rx, f.kx);
        }
    }
}

// ... then the outputs, and partial column sums: a thread owns one vector of columns.
// Parts lie within the rows of a gate row; blockIdx.y takes every gridDim.y-th, and
// keeps one sum of dpre_w over all of them.
template <typename T, int VB>
__global__ void __launch_bounds__(kBlockColsThreads) blocknorm_bwd_cols_kernel(const BlockParams p) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x * kBlockColsThreads + threadIdx.x;
    if (i >= p.nvec) return;
    const int64_t row_bytes = static_cast<int64_t>(p.hidden) * sizeof(T);
    const int64_t col = static_cast<int64_t>(i) * VB;
    float pw[EPV], sw[EPV], pre[EPV];
    widen_ro<T, VB>(pw, at_or_null(p.pre_w, col));
    widen_ro<T, VB>(sw, at_or_null(p.post ? p.post_w : nullptr, col));
#pragma unroll
    for (int k = 0; k < EPV; ++k) pre[k] = 0.f;
    for (int64_t part = blockIdx.y; part < p.parts; part += gridDim.y) {
        const int64_t s = part / p.parts_per_gate;
        const int64_t r0 = s * p.gate_rows + part % p.parts_per_gate * p.rows_per_part;
        int64_t r1 = r0 + p.rows_per_part;
        if (r1 > (s + 1) * p.gate_rows) r1 = (s + 1) * p.gate_rows;
        if (r1 > p.rows) r1 = p.rows;
        float u[EPV], acc[EPV];
        widen_ro<T, VB>(u, at_or_null(p.gate, s * row_bytes + col));
#pragma unroll
        for (int k = 0; k < EPV; ++k) {
            u[k] *= sw[k];
            acc[k] = 0.f;
        }
        for (int64_t row = r0; row < r1; ++row) {
            const int64_t at = row * row_bytes + col;
            const float4 f = p.row_stats[row];
            const Vec<VB> xv = ld_plain<VB>(static_cast<const char*>(p.x) + at);
            float d[EPV], dx[EPV], dr[EPV];
#pragma unroll
            for (int k = 0; k < EPV; ++k) d[k] = 0.f;
            if (p.dh) {
                const Vec<VB> dv = ld_plain<VB>(static_cast<const char*>(p.dh) + at);
#pragma unroll
                for (int k = 0; k < EPV; ++k) d[k] = get<T, VB>(dv, k);
            }
            if (p.pre) {
                const Vec<VB> yv = ld_plain<VB>(static_cast<const char*>(p.dy) + at);
                const Vec<VB> hv = ld_plain<VB>(static_cast<const char*>(p.h_in) + at);
#pragma unroll
                for (int k = 0; k < EPV; ++k) {
                    const float h = get<T, VB>(hv, k), dy = get<T, VB>(yv, k);
                    pre[k] = fmaf(dy, h * f.x, pre[k]);
                    d[k] = fmaf(f.x, fmaf(dy, pw[k], -(h * f.y)), d[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < EPV; ++k) {
                const float x = get<T, VB>(xv, k);
                acc[k] = fmaf(d[k], x * f.z, acc[k]);
                const float e = p.branch_scale * d[k] * u[k];
                dx[k] = p.post ? f.z * (e - x * f.w) : e;     // an infinite x * 0 is not 0
                dr[k] = p.residual_scale * d[k];
            }
            st_stream<VB>(static_cast<char*>(p.dx) + at, pack<T, VB>(dx));
            st_stream<VB>(static_cast<char*>(p.dres) + at, pack<T, VB>(dr));
        }
        if (p.part_gate) {
            float* to = p.part_gate + part * p.hidden + static_cast<int64_t>(i) * EPV;
#pragma unroll
            for (int k = 0; k < EPV; ++k) to[k] = acc[k];
        }
    }
    if (p.part_pre) {
        float* to = p.part_pre + static_cast<int64_t>(blockIdx.y) * p.hidden + static_cast<int64_t>(i) * EPV;
#pragma unroll
        for (int k = 0; k < EPV; ++k) to[k] = pre[k];
    }
}

// ----------------------------------------------------------- sums over parts --
//
// A CTA takes 8 * W columns, of which each of its 32 lanes adds every 32nd part, ten
// loads in flight, then the lanes in order (as the norm backward passes' sums).
// Gate row s has A[s] = the sum of its parts:
//   dgate[s] = branch_scale * post_w * A[s],   dpost_w = branch_scale * sum_s gate[s] * A[s]
// With one gate row both come from here; with several A is kept, and dpost_w
// is formed from it by a second launch (GATES false).  Where the gate rows have few parts
// each, lanes for 32 parts would be idle (32 gate rows of 5 parts, 8192 wide: 38 us), and a
// thread adds its columns' by itself.

template <int W>
__device__ __forceinline__ void load_cols(float (&v)[W], const float* from) {
    if constexpr (W == 4) {
        const float4 f = *reinterpret_cast<const float4*>(from);
        v[0] = f.x;
        v[1] = f.y;
        v[2] = f.z;
        v[3] = f.w;
    } else {
        v[0] = *from;
    }
}

// Sum over `count` parts of the CTA's columns; `weigh` (count rows of T) multiplies
// them if it is given.  The threads below COLS * W have the sum of column
// blockIdx.x * COLS * W + threadIdx.x.
template <typename T, int W>
__device__ __forceinline__ float sum_parts(const float* part, int64_t count, int hidden,
                                           const T* weigh) {
    constexpr int COLS = kBlockReduceCols, LANES = kBlockReduceThreads / COLS, U = 10;
    __shared__ float red[kBlockReduceThreads / 32][COLS * W];
    const int c = threadIdx.x % COLS, l = threadIdx.x / COLS;
    int64_t col = (static_cast<int64_t>(blockIdx.x) * COLS + c) * W;
    if (col >= hidden) col = 0;                  // read again, not written
    float s[W];
#pragma unroll
    for (int w = 0; w < W; ++w) s[w] = 0.f;
    for (int64_t k = l; k < count; k += U * LANES) {
        float v[U][W];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // loads past the last part repeat it and are not added
            const int64_t at = min(k + u * LANES, count - 1) * hidden + col;
            load_cols<W>(v[u], part + at);
            if (weigh) {
#pragma unroll
                for (int w = 0; w < W; ++w) v[u][w] *= static_cast<float>(weigh[at + w]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k + u * LANES < count) {
#pragma unroll
                for (int w = 0; w < W; ++w) s[w] += v[u][w];
            }
        }
    }
    __syncthreads();                             // the last call's sums have been read
#pragma unroll
    for (int w = 0; w < W; ++w) {
#pragma unroll
        for (int m = COLS; m < 32; m <<= 1) s[w] += __shfl_xor_sync(0xffffffffu, s[w], m);
        if ((threadIdx.x & 31) < COLS) red[threadIdx.x >> 5][c * W + w] = s[w];
    }
    __syncthreads();
    float v = 0.f;
    if (threadIdx.x < COLS * W) {
#pragma unroll
        for (int k = 0; k < kBlockReduceThreads / 32; ++k) v += red[k][threadIdx.x];
    }
    return v;
}

template <typename T, int W, bool GATES>
__global__ void __launch_bounds__(kBlockReduceThreads) blocknorm_reduce_kernel(const BlockParams p) {
    pdl_trigger();
    pdl_wait();
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kBlockReduceCols * W + threadIdx.x;
    const bool mine = threadIdx.x < kBlockReduceCols * W && col < p.hidden;
    const T* gate = static_cast<const T*>(p.gate);
    if constexpr (!GATES) {
        const float v = sum_parts<T, W>(p.gate_sums, p.gates, p.hidden, gate);
        if (mine) p.dpost_w[col] = p.branch_scale * v;
        return;
    }
    if (blockIdx.y == 0) {
        if (!p.part_pre) return;
        const float v = sum_parts<T, W>(p.part_pre, p.pre_parts, p.hidden, nullptr);
        if (mine) p.dpre_w[col] = v;
        return;
    }
    if (!p.part_gate) return;
    const T* post_w = p.post ? static_cast<const T*>(p.post_w) : nullptr;
    auto parts_of = [&](int64_t s, int64_t& from, int64_t& count) {
        from = s * p.parts_per_gate;
        count = p.parts_per_gate;
        if (p.units && p.gates == 1) {
            count = p.units;
        } else if (p.units) {   // the units that the gate row's blocks were dealt to
            const int64_t b0 = s * p.blocks_per_gate;
            const int64_t b1 = min(b0 + p.blocks_per_gate, p.blocks) - 1;
            const int64_t u0 = div_nonneg((b0 + 1) * p.units - 1, p.blocks);
            from = u0 + s;
            count = div_nonneg((b1 + 1) * p.units - 1, p.blocks) - u0 + 1;
        }
    };
    if (p.few_parts) {          // a thread for W columns of a gate row
        const int64_t per_gate = (p.hidden + kBlockReduceThreads * W - 1) / (kBlockReduceThreads * W);
        const int64_t ctas = static_cast<int64_t>(gridDim.x) * (gridDim.y - 1);
        for (int64_t task = blockIdx.x + static_cast<int64_t>(gridDim.x) * (blockIdx.y - 1);
             task < per_gate * p.gates; task += ctas) {
            const int64_t s = div_nonneg(task, per_gate);
            const int64_t c = ((task - s * per_gate) * kBlockReduceThreads + threadIdx.x) * W;
            if (c >= p.hidden) continue;
            int64_t from, count;
            parts_of(s, from, count);
            float v[W];
#pragma unroll
            for (int w = 0; w < W; ++w) v[w] = 0.f;
            for (int64_t k = 0; k < count; k += 4) {
                float f[4][W];
#pragma unroll
                for (int u = 0; u < 4; ++u)      // past the last part it again, not added
                    load_cols<W>(f[u], p.part_gate + (from + min(k + u, count - 1)) * p.hidden + c);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (k + u < count) {
#pragma unroll
                        for (int w = 0; w < W; ++w) v[w] += f[u][w];
                    }
                }
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int64_t at = s * p.hidden + c + w;
                if (p.dgate)
                    p.dgate[at] = p.branch_scale * v[w] * (post_w ? static_cast<float>(post_w[c + w]) : 1.f);
                if (p.gate_sums) p.gate_sums[at] = v[w];
            }
        }
        return;
    }
    for (int64_t s = blockIdx.y - 1; s < p.gates; s += gridDim.y - 1) {
        int64_t from, count;
        parts_of(s, from, count);
        const float v = sum_parts<T, W>(p.part_gate + from * p.hidden, count, p.hidden, nullptr);
        if (!mine) continue;
        const int64_t at = s * p.hidden + col;
        if (p.dgate) p.dgate[at] = p.branch_scale * v * (post_w ? static_cast<float>(post_w[col]) : 1.f);
        if (p.gates > 1) {
            if (p.gate_sums) p.gate_sums[at] = v;
        } else if (p.dpost_w) {
            p.dpost_w[col] = p.branch_scale * v * (gate ? static_cast<float>(gate[col]) : 1.f);
        }
    }
}

}  // namespace rmsnorm
