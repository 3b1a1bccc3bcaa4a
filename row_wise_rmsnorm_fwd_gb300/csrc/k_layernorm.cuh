// k_layernorm.cuh -- layer norm forward.
//
//     mean = (1/H) sum_j x[j]     var = (1/H) sum_j (x[j] - mean)^2
//     y[j] = (x[j] - mean) * rsqrt(var + eps) * w[j] + b[j]
//
// The variance is never formed as a difference of large sums: elements are
// taken in small groups, each with its own mean and sum of squares about that
// mean, and groups are merged by the pairwise update
//     M2 = M2a + M2b + (mean_b - mean_a)^2 * na * nb / (na + nb)
// (Chan, Golub and LeVeque, "Updating formulae and a pairwise algorithm for
// computing sample variances", 1979), so a row whose mean is far larger than
// its spread loses nothing but the rounding of its own elements.
#pragma once
#include "common.cuh"
#include "norm_launch.h"

namespace rmsnorm {

struct Moments {
    float n, mean, m2;     // count, mean, sum of squares about the mean
};

__device__ __forceinline__ void merge(Moments& a, const Moments& b) {
    const float n = a.n + b.n;
    const float f = n > 0.f ? b.n / n : 0.f;
    const float d = b.mean - a.mean;
    a.m2 += b.m2 + d * d * a.n * f;
    a.mean += d * f;
    a.n = n;
}

// Butterfly over the warp; all lanes end with the same bits (the merge is
// evaluated with the lower lane's value first on both sides).
__device__ __forceinline__ Moments warp_merge(Moments a) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        Moments o;
        o.n = __shfl_xor_sync(0xffffffffu, a.n, m);
        o.mean = __shfl_xor_sync(0xffffffffu, a.mean, m);
        o.m2 = __shfl_xor_sync(0xffffffffu, a.m2, m);
        if (lane & m) {
            merge(o, a);
            a = o;
        } else {
            merge(a, o);
        }
    }
    return a;
}

// Any width and alignment: one CTA per row, which reads the row twice (the
// second read normally from L2).
constexpr int kLayerTwopassThreads = 512;
constexpr int kLayerTwopassGroup = 4;      // vectors merged at a time

template <typename T, int VB>
__global__ void __launch_bounds__(kLayerTwopassThreads)
layernorm_twopass_kernel(const NormParams p) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    constexpr int U = kLayerTwopassGroup;
    __shared__ Moments red[kLayerTwopassThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nwarp = blockDim.x >> 5;
    const char* wb = static_cast<const char*>(p.w);
    const char* bb = static_cast<const char*>(p.b);
    const int64_t row_bytes = static_cast<int64_t>(p.hidden) * sizeof(T);

    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const char* src = static_cast<const char*>(p.x) + row * row_bytes;
        char* dst = static_cast<char*>(p.out) + row * row_bytes;
        Moments acc{0.f, 0.f, 0.f};
        for (int64_t v0 = tid; v0 < p.nvec; v0 += static_cast<int64_t>(U) * blockDim.x) {
            Vec<VB> v[U];
            int cnt = 0;
            float s = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = v0 + static_cast<int64_t>(u) * blockDim.x;
                if (i < p.nvec) {
                    v[u] = ld_plain<VB>(src + i * VB);
                    cnt += EPV;
#pragma unroll
                    for (int k = 0; k < EPV; ++k) s += get<T, VB>(v[u], k);
                }
            }
            Moments g;
            g.n = static_cast<float>(cnt);
            g.mean = s / g.n;
            g.m2 = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (v0 + static_cast<int64_t>(u) * blockDim.x < p.nvec) {
#pragma unroll
                    for (int k = 0; k < EPV; ++k) {
                        const float d = get<T, VB>(v[u], k) - g.mean;
                        g.m2 = fmaf(d, d, g.m2);
                    }
                }
            }
            merge(acc, g);
        }
        acc = warp_merge(acc);
        if (lane == 0) red[warp] = acc;
        __syncthreads();
        acc = red[0];
        for (int k = 1; k < nwarp; ++k) merge(acc, red[k]);
        const float mean = acc.mean;
        const float rstd = rsqrtf(fmaf(acc.m2, p.inv_hidden, p.eps));
        if (tid == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        for (int64_t i = tid; i < p.nvec; i += blockDim.x) {
            const Vec<VB> v = ld_plain<VB>(src + i * VB);
            Vec<VB> wv, bv;
            if (wb) wv = ld_ro<VB>(wb + i * VB);
            if (bb) bv = ld_ro<VB>(bb + i * VB);
            float o[EPV];
#pragma unroll
            for (int k = 0; k < EPV; ++k) {
                const float xh = (get<T, VB>(v, k) - mean) * rstd;
                const float wk = wb ? get<T, VB>(wv, k) : 1.f;
                const float bk = bb ? get<T, VB>(bv, k) : 0.f;
                o[k] = fmaf(xh, wk, bk);
            }
            st_stream<VB>(dst + i * VB, pack<T, VB>(o));
        }
        __syncthreads();        // red[] is written again for the next row
    }
}

}  // namespace rmsnorm
