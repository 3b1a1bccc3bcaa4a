// k_normbwd.cuh -- backward passes of layer norm and RMSNorm.
//
// With xh the normalised row, g = dy * w and m(.) the mean over a row:
//   layer norm  xh = (x - mean) * rstd (mean and rstd from the forward pass)
//               dx = rstd * (g - m(g) - xh * m(g * xh))
//   RMSNorm     rstd = rsqrt(m(x^2) + eps), xh = x * rstd
//               dx = rstd * (g - xh * m(g * xh))
//   both        dw = sum over rows of dy * xh;  layer norm: db = sum of dy
//
// Column sums are kept in fp32 per part (a fixed set of rows) and the parts
// are added in a fixed order by a last kernel: no atomics, so results are
// bitwise repeatable.
#pragma once
#include "common.cuh"
#include "norm_launch.h"

namespace rmsnorm {

// Sum a pair over the block (at most 32 warps); all threads get the same bits.
// red: 32 slots, free again after the caller's next barrier.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* red) {
    a = warp_allreduce_sum(a);
    b = warp_allreduce_sum(b);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
    const int n = blockDim.x >> 5;
    for (int k = 0; k < n; ++k) {
        s.x += red[k].x;
        s.y += red[k].y;
    }
    return s;
}

// ------------------------------------------- any width: three kernels --

constexpr int kBwdRowsThreads = 256;
constexpr int kBwdColsThreads = 128;

// The pair of each row: layer norm (m(g), m(g * xh)), RMSNorm (rstd, m(g * xh)).
template <typename T, int VB, bool LAYER>
__global__ void __launch_bounds__(kBwdRowsThreads) norm_bwd_rows_kernel(const NormParams p) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    __shared__ float2 red[2][32];
    pdl_trigger();
    pdl_wait();
    const char* wb = static_cast<const char*>(p.w);
    const int64_t row_bytes = static_cast<int64_t>(p.hidden) * sizeof(T);
    int it = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, ++it) {
        const char* xs = static_cast<const char*>(p.x) + row * row_bytes;
        const char* ds = static_cast<const char*>(p.dy) + row * row_bytes;
        const float mean = LAYER ? p.mean[row] : 0.f;
        const float rstd = LAYER ? p.rstd[row] : 1.f;
        float a = 0.f, b = 0.f;
        for (int64_t i = threadIdx.x; i < p.nvec; i += kBwdRowsThreads) {
            const Vec<VB> xv = ld_plain<VB>(xs + i * VB);
            const Vec<VB> dv = ld_plain<VB>(ds + i * VB);
            Vec<VB> wv;
            if (wb) wv = ld_ro<VB>(wb + i * VB);
            float va = 0.f, vb = 0.f;
#pragma unroll
            for (int k = 0; k < EPV; ++k) {
                const float x = get<T, VB>(xv, k);
                const float g = get<T, VB>(dv, k) * (wb ? get<T, VB>(wv, k) : 1.f);
                const float xh = LAYER ? (x - mean) * rstd : x;
                va = LAYER ? va + g : fmaf(x, x, va);
                vb = fmaf(g, xh, vb);
            }
            a += va;
            b += vb;
        }
        const float2 s = block_sum2(a, b, red[it & 1]);
        if (threadIdx.x == 0) {
            float2 o;
            if (LAYER) {
                o = make_float2(s.x * p.inv_hidden, s.y * p.inv_hidden);
            } else {
                o.x = rsqrtf(fmaf(s.x, p.inv_hidden, p.eps));
                o.y = s.y * o.x * p.inv_hidden;
            }
            p.row_stats[row] = o;
        }
    }
}

// dx, and the partial column sums of rows [part * rows_per_part, ...): a
// thread owns one vector of columns, blockIdx.y is the part.
template <typename T, int VB, bool LAYER>
__global__ void __launch_bounds__(kBwdColsThreads) norm_bwd_cols_kernel(const NormParams p) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    pdl_trigger();
    pdl_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kBwdColsThreads + threadIdx.x;
    if (i >= p.nvec) return;
    const int64_t row_bytes = static_cast<int64_t>(p.hidden) * sizeof(T);
    float w[EPV], aw[EPV], ab[EPV];
#pragma unroll
    for (int k = 0; k < EPV; ++k) {
        w[k] = 1.f;
        aw[k] = ab[k] = 0.f;
    }
    if (p.w) {
        const Vec<VB> wv = ld_ro<VB>(static_cast<const char*>(p.w) + i * VB);
#pragma unroll
        for (int k = 0; k < EPV; ++k) w[k] = get<T, VB>(wv, k);
    }
    const int64_t r0 = blockIdx.y * p.rows_per_part;
    const int64_t r1 = min(p.rows, r0 + p.rows_per_part);
#pragma unroll 2
    for (int64_t row = r0; row < r1; ++row) {
        const int64_t at = row * row_bytes + i * VB;
        const Vec<VB> xv = ld_plain<VB>(static_cast<const char*>(p.x) + at);
        const Vec<VB> dv = ld_plain<VB>(static_cast<const char*>(p.dy) + at);
        const float2 st = p.row_stats[row];
        const float mean = LAYER ? p.mean[row] : 0.f;
        const float rstd = LAYER ? p.rstd[row] : st.x;
        const float c1 = LAYER ? st.x : 0.f;
        float o[EPV];
#pragma unroll
        for (int k = 0; k < EPV; ++k) {
            const float dy = get<T, VB>(dv, k);
            const float xh = (get<T, VB>(xv, k) - mean) * rstd;
            aw[k] = fmaf(dy, xh, aw[k]);
            if (LAYER) ab[k] += dy;
            o[k] = rstd * (fmaf(dy, w[k], -c1) - xh * st.y);
        }
        st_stream<VB>(static_cast<char*>(p.out) + at, pack<T, VB>(o));
    }
    const int64_t at = static_cast<int64_t>(blockIdx.y) * p.hidden + i * EPV;
#pragma unroll
    for (int k = 0; k < EPV; ++k) {
        if (p.part_w) p.part_w[at + k] = aw[k];
        if (LAYER && p.part_b) p.part_b[at + k] = ab[k];
    }
}

// dw and db from the parts: a CTA takes 32 columns, its 16 rows of threads
// every 16th part each, then their sums in order.  grid.y: 0 = dw, 1 = db.
static __global__ void __launch_bounds__(kNormReduceCols * kNormReduceLanes)
norm_bwd_reduce_kernel(const NormParams p) {
    __shared__ float red[kNormReduceLanes][kNormReduceCols + 1];
    pdl_trigger();
    pdl_wait();
    const int c = threadIdx.x % kNormReduceCols, l = threadIdx.x / kNormReduceCols;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kNormReduceCols + c;
    const float* part = blockIdx.y ? p.part_b : p.part_w;
    float* out = blockIdx.y ? p.db : p.dw;
    if (!part) return;
    float s = 0.f;
    if (col < p.hidden) {
#pragma unroll 4
        for (int k = l; k < p.parts; k += kNormReduceLanes)
            s += part[static_cast<int64_t>(k) * p.hidden + col];
    }
    red[l][c] = s;
    __syncthreads();
    if (l == 0 && col < p.hidden) {
        s = 0.f;
        for (int k = 0; k < kNormReduceLanes; ++k) s += red[k][c];
        out[col] = s;
    }
}

}  // namespace rmsnorm
