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
#include "k_blockring.cuh"
#include "norm_launch.h"
#include "pairs.cuh"

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

// Rows staged in shared memory by bulk copies (k_blockring.cuh): blocks of
// p.rows_per_cta rows, G threads per row (p.group: a multiple of 32, or a power
// of two below 32 for several rows per warp); x is read from HBM once and from
// shared memory three times (sum, squares, output), which costs no registers,
// so bf16 rows, which are bound by the issue slots rather than by HBM, run
// with nothing but their arithmetic, on packed pairs.  Each warp (lane group)
// forms the mean of its own share of a row and the squares about it, and one
// exchange through shared memory, behind one barrier, merges the warps' pairs:
// the merge update above, for shares of fixed counts, with the row's mean
// known first.
template <typename T, int VB>
__global__ void __launch_bounds__(1024) layernorm_staged_kernel(const NormParams p) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    constexpr int PN = PairTraits<T, VB>::N;
    using L = Lanes<PairTraits<T, VB>::W>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ alignas(8) uint64_t bars[kBlockRingMaxSlots];
    __shared__ float2 red[2][32];
    pdl_trigger();
    const int G = p.group;
    const int width = G < 32 ? G : 32;       // lanes of a share
    const int tid = threadIdx.x;
    const int g = tid / G;
    const int t = tid - g * G;
    const int warp = tid >> 5, lane = tid & 31;
    const int wpg = G >> 5;
    const int gw0 = g * wpg;
    const int rpc = p.rows_per_cta;
    const int row_bytes = p.hidden * static_cast<int>(sizeof(T));

    BlockRing ring;
    ring.nslots = p.nslots;
    ring.slot_bytes = p.slot_bytes;
    ring.block_bytes = static_cast<int64_t>(rpc) * row_bytes;
    ring.total_bytes = p.rows * row_bytes;
    ring.init(p.x, nullptr, smem, bars, (p.rows + rpc - 1) / rpc);
    // elements of this share of a row, and of the share that lane k < wpg merges
    auto share_of = [&](int w) {
        int n = 0;
        for (int v = w * 32; v < p.nvec; v += G) n += min(32, p.nvec - v);
        return static_cast<float>(n * EPV);
    };
    const float cnt = wpg > 1 ? share_of(warp - gw0) : static_cast<float>(p.hidden);
    const float inv_cnt = cnt > 0.f ? 1.f / cnt : 0.f;
    const float cnt_k = wpg > 1 && lane < wpg ? share_of(lane) : 0.f;
    const float inv_k = cnt_k > 0.f ? 1.f / cnt_k : 0.f;
    int merge_width = 1;
    while (merge_width < wpg) merge_width <<= 1;
    const int full = p.nvec / G;
    const bool more = t < p.nvec - full * G;
    __syncthreads();
    pdl_wait();
    if (tid == 0) ring.prologue(p.fault);

    const char* wb = static_cast<const char*>(p.w);
    const char* bb = static_cast<const char*>(p.b);
    int64_t row = static_cast<int64_t>(blockIdx.x) * rpc + g;
    const int64_t row_step = static_cast<int64_t>(gridDim.x) * rpc;
    RingStep step;
    int n = 0;
    for (; n < ring.count; ++n, row += row_step) {
        const bool ok = ring.wait(step, p.timeout_ns);
        if (n >= ring.tail_from) ring.finish<T>(step.slot, n);
        const uint32_t src = ring.base(step.slot, 0) + static_cast<uint32_t>(ring.start(n) & 15) +
                             static_cast<uint32_t>(g * row_bytes);

        L s0 = L::all(0.f), s1 = L::all(0.f);
        for_vectors(t, G, full, more, [&](int v) {
            const Vec<VB> x = ld_slot<VB>(src + v * VB);
#pragma unroll
            for (int k = 0; k < PN; ++k) {
                if (k & 1) s1 = lanes_plus<T, VB>(x, k, s1); else s0 = lanes_plus<T, VB>(x, k, s0);
            }
        });
        const float sum = share_sum((s0 + s1).total(), width);
        const float part = sum * inv_cnt;            // mean of the share
        const L about = L::all(-part);
        s0 = s1 = L::all(0.f);
        for_vectors(t, G, full, more, [&](int v) {
            const Vec<VB> x = ld_slot<VB>(src + v * VB);
#pragma unroll
            for (int k = 0; k < PN; ++k) {
                const L d = lanes_plus<T, VB>(x, k, about);
                if (k & 1) s1 = fma(d, d, s1); else s0 = fma(d, d, s0);
            }
        });
        float m2 = share_sum((s0 + s1).total(), width);
        float mean = part;
        float2* slot = red[n & 1];
        if (wpg > 1 && lane == 0) slot[warp] = make_float2(sum, m2);
        if (__syncthreads_or(!ok)) break;            // uniform; also frees the previous slot
        if (tid == 0) ring.refill(step, n, p.fault);
        if (wpg > 1) {
            float2 e = make_float2(0.f, 0.f);
            if (lane < wpg) e = slot[gw0 + lane];
            mean = group_allreduce_sum(e.x, merge_width);
            mean = __shfl_sync(0xffffffffu, mean, 0) * p.inv_hidden;
            // n_k * (mean_k - mean)^2, from the share's sum and count
            const float d = fmaf(-cnt_k, mean, e.x);
            m2 = group_allreduce_sum(fmaf(d * inv_k, d, e.y), merge_width);
            m2 = __shfl_sync(0xffffffffu, m2, 0);
        }
        const float rstd = rsqrtf(fmaf(m2, p.inv_hidden, p.eps));
        if (row < p.rows) {
            if (t == 0) {
                if (p.mean) p.mean[row] = mean;
                if (p.rstd) p.rstd[row] = rstd;
            }
            char* dst = static_cast<char*>(p.out) + row * row_bytes;
            const L minus = L::all(-mean), r = L::all(rstd);
            auto write = [&](auto with_w, auto with_b) {
                for_vectors(t, G, full, more, [&](int v) {
                    const Vec<VB> x = ld_slot<VB>(src + v * VB);
                    Vec<VB> wi, bi;
                    if constexpr (with_w) wi = ld_ro<VB>(wb + v * VB);
                    if constexpr (with_b) bi = ld_ro<VB>(bb + v * VB);
                    float o[EPV];
#pragma unroll
                    for (int k = 0; k < PN; ++k) {
                        L y = lanes_plus<T, VB>(x, k, minus) * r;
                        if constexpr (with_w && with_b) {
                            y = fma(y, lanes<T, VB>(wi, k), lanes<T, VB>(bi, k));
                        } else if constexpr (with_w) {
                            y = y * lanes<T, VB>(wi, k);
                        } else if constexpr (with_b) {
                            y = y + lanes<T, VB>(bi, k);
                        }
                        y.put(o + k * (EPV / PN));
                    }
                    st_stream<VB>(dst + v * VB, pack<T, VB>(o));
                });
            };
            using Yes = std::true_type;
            using No = std::false_type;
            if (wb) {
                if (bb) write(Yes(), Yes()); else write(Yes(), No());
            } else {
                if (bb) write(No(), Yes()); else write(No(), No());
            }
        }
        step.next(ring.nslots);
    }
    if (n < ring.count) {
        // a wait ran out: report it, and let the copies that are under way land
        if (tid == 0) {
            report_timeout(p.status, kSiteStagedFull);
            ring.drain(step, n, p.timeout_ns);
        }
        __syncthreads();
    }
}

}  // namespace rmsnorm
