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
// computing sample variances", 1979), so the variance of a row whose mean is far
// larger than its spread is as good as any other's.  The mean itself is as good as
// an fp32 sum: off by the rounding of its additions, and exact where they are.
#pragma once
#include "common.cuh"
#include "k_blockring.cuh"
#include "norm_launch.h"
#include "pairs.cuh"

namespace rmsnorm {

// sum / count by the count's reciprocal, whose rounding is taken back out: without
// that a constant row at a width that has no exact reciprocal is off its own mean
// by 2^-23 of it, which rstd may make any size.  An infinite sum stays.  Two divisions
// a row instead: bf16 65536 x 4096 182 us against 174.
__device__ __forceinline__ float mean_of(float sum, float count, float inv) {
    const float m = sum * inv;
    const float rest = fmaf(-count, m, sum);
    return fabsf(rest) < INFINITY ? fmaf(rest, inv, m) : m;
}

struct Moments {
    float n, mean, m2;     // count, mean, sum of squares about the mean
};

__device__ __forceinline__ void merge(Moments& a, const Moments& b) {
    const float n = a.n + b.n;
    const float f = n > 0.f ? b.n / n : 0.f;
    const float d = b.mean - a.mean;
    // nothing where one of the two is empty: its mean of 0 may be so far away that
    // the square of the distance is infinite
    a.m2 += b.m2 + (a.n > 0.f && b.n > 0.f ? d * d * a.n * f : 0.f);
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
// second read normally from L2).  Two dependent reads with a block barrier
// between them bound it: a third of the HBM copy peak for fp32 rows of 4096, a
// sixth for bf16; it takes what the staged kernel below cannot.
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

// Rows staged in shared memory by bulk copies (k_blockring.cuh; SHIFT: rows of
// any length, the weights copied to shared memory in their layout): blocks of
// p.rows_per_cta rows, G threads per row (p.group: a multiple of 32, or a power
// of two below 32 for several rows per warp); x is read from HBM once and from
// shared memory three times (sum, squares, output), which costs no registers,
// so bf16 rows, which are bound by the issue slots rather than by HBM, run
// with nothing but their arithmetic, on packed pairs.  Each warp (lane group)
// forms the mean of its own share of a row and the squares about it, and one
// exchange through shared memory, behind one barrier, merges the warps' pairs:
// the merge update above, for shares of fixed counts, with the row's mean
// known first.
//
// Measured (launches back to back, % of the HBM copy peak): fp32 65536 x 4096 323 us,
// 98, bound by HBM; bf16 65536 x 8192 338 us, 94, 65536 x 1024 48 us, 82: half as many
// bytes for the same instructions.  Rows of any length, whose edges are stored
// element by element: bf16 16384 x 4097 64 us, 62, 8191 x 2050 21.6 us, 46.  Reading
// the row twice instead (above): 954 and, bf16 65536 x 4096, 938 us against 173.
template <typename T, bool SHIFT>
__global__ void __launch_bounds__(1024) layernorm_staged_kernel(const NormParams p) {
    constexpr int EPV = VecTraits<T, 16>::kElems;
    constexpr int PN = kPairs<T>;
    using L = Lanes;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ alignas(8) uint64_t bars[kBlockRingMaxSlots];
    __shared__ float2 red[2][32];
    __shared__ float2 count[32];             // elements of a warp's share, and 1 / that
    pdl_trigger();
    const int G = p.group;
    const int width = G < 32 ? G : 32;       // lanes of a share
    const int tid = threadIdx.x;
    const int g = tid / G;
    const int t = tid - g * G;
    const int warp = tid >> 5, lane = tid & 31;
    const int wpg = G >> 5;
    const int gw0 = g * wpg;

    const RowRing<T, SHIFT, 1> ring(p, p.rows_per_cta, smem, bars);
    const RowVecs<T, SHIFT> rv(ring.shift, p.hidden);
    const int full = rv.nvec / G;
    const bool more = t < rv.nvec - full * G;
    // elements of this share of a row, and of the share that lane k < wpg merges
    int mine = 0;
    for_vectors(t, G, full, more, [&](int) { mine += EPV; });
    for (int e = t; e < rv.edges; e += G) ++mine;
    const float cnt = share_sum(static_cast<float>(mine), width);
    const float inv_cnt = 1.f / cnt;                 // every share has an element
    if (wpg > 1 && lane == 0) count[warp] = make_float2(cnt, inv_cnt);
    int merge_width = 1;
    while (merge_width < wpg) merge_width <<= 1;
    __syncthreads();
    float2 share = make_float2(0.f, 0.f);
    if (wpg > 1 && lane < wpg) share = count[gw0 + lane];
    pdl_wait();
    if (warp == 0) ring.prologue();

    // the weights: in global memory, or laid out like the rows behind the ring
    const char* wg = static_cast<const char*>(p.w);
    const char* bg = static_cast<const char*>(p.b);
    uint32_t ws = 0, bs = 0;
    if constexpr (SHIFT) {
        T* wc = reinterpret_cast<T*>(smem + (ring.base(p.nslots, 0) - ring.base(0, 0)));
        const int size = ring.row_slot() / static_cast<int>(sizeof(T));
        T* bc = wc + size;
        copy_shifted<T>(wc, p.w, rv.skip, p.hidden, size, 1.f);
        copy_shifted<T>(bc, p.b, rv.skip, p.hidden, size, 0.f);
        ws = smem_addr(wc);
        bs = smem_addr(bc);
        // read behind the first iteration's barrier
    }
    int64_t row = ring.first + static_cast<int64_t>(g) * ring.period();
    RingStep step;
    int n = 0;
    for (; n < ring.count; ++n, row += ring.step) {
        const bool ok = ring.wait(step);
        ring.finish(step.slot, n);
        const uint32_t in_slot = ring.base(step.slot, 0) + static_cast<uint32_t>(g * ring.row_slot());
        const uint32_t src = in_slot + static_cast<uint32_t>(rv.vec_at());

        L s0 = L::all(0.f), s1 = L::all(0.f);
        for_vectors(t, G, full, more, [&](int v) {
            const Vec<16> x = ld_slot(src + v * 16);
#pragma unroll
            for (int k = 0; k < PN; ++k) {
                if (k & 1) s1 = lanes_plus<T>(x, k, s1); else s0 = lanes_plus<T>(x, k, s0);
            }
        });
        float sum = (s0 + s1).total();
        if constexpr (SHIFT)
            for (int e = t; e < rv.edges; e += G) sum += ld_elem<T>(in_slot + rv.edge_at(e));
        sum = share_sum(sum, width);
        // mean of the share; SHIFT has no register for the reciprocal (fp32 16384 x 4097
        // 119 us, by the reciprocal 137)
        const float part = SHIFT ? sum / cnt : mean_of(sum, cnt, inv_cnt);
        const L about = L::all(-part);
        s0 = s1 = L::all(0.f);
        for_vectors(t, G, full, more, [&](int v) {
            const Vec<16> x = ld_slot(src + v * 16);
#pragma unroll
            for (int k = 0; k < PN; ++k) {
                const L d = lanes_plus<T>(x, k, about);
                if (k & 1) s1 = fma(d, d, s1); else s0 = fma(d, d, s0);
            }
        });
        float m2 = (s0 + s1).total();
        if constexpr (SHIFT) {
            for (int e = t; e < rv.edges; e += G) {
                const float d = ld_elem<T>(in_slot + rv.edge_at(e)) - part;
                m2 = fmaf(d, d, m2);
            }
        }
        m2 = share_sum(m2, width);
        float mean = part;
        float2* slot = red[n & 1];
        if (wpg > 1 && lane == 0) slot[warp] = make_float2(sum, m2);
        if (__syncthreads_or(!ok)) break;            // uniform; also frees the previous slot
        if (warp == 0) ring.refill(step, n);
        if (wpg > 1) {
            float2 e = make_float2(0.f, 0.f);
            if (lane < wpg) e = slot[gw0 + lane];
            mean = group_allreduce_sum(e.x, merge_width);
            mean = mean_of(__shfl_sync(0xffffffffu, mean, 0), static_cast<float>(p.hidden),
                           p.inv_hidden);
            // n_k * (mean_k - mean)^2, from the share's sum and count
            const float d = fmaf(-share.x, mean, e.x);
            m2 = group_allreduce_sum(fmaf(d * share.y, d, e.y), merge_width);
            m2 = __shfl_sync(0xffffffffu, m2, 0);
        }
        const float rstd = rsqrtf(fmaf(m2, p.inv_hidden, p.eps));
        if (row < p.rows) {
            if (t == 0) {
                if (p.mean) p.mean[row] = mean;
                if (p.rstd) p.rstd[row] = rstd;
            }
            const int64_t at = row * p.hidden;
            char* dst = static_cast<char*>(p.out) + (at + rv.head) * static_cast<int>(sizeof(T));
            const L minus = L::all(-mean), r = L::all(rstd);
            auto write = [&](auto with_w, auto with_b) {
                for_vectors(t, G, full, more, [&](int v) {
                    const Vec<16> x = ld_slot(src + v * 16);
                    Vec<16> wi, bi;
                    if constexpr (with_w)
                        wi = SHIFT ? ld_slot(ws + rv.vec_at() + v * 16) : ld_ro<16>(wg + v * 16);
                    if constexpr (with_b)
                        bi = SHIFT ? ld_slot(bs + rv.vec_at() + v * 16) : ld_ro<16>(bg + v * 16);
                    float o[EPV];
#pragma unroll
                    for (int k = 0; k < PN; ++k) {
                        L y = lanes_plus<T>(x, k, minus) * r;
                        if constexpr (with_w && with_b) {
                            y = fma(y, lanes<T>(wi, k), lanes<T>(bi, k));
                        } else if constexpr (with_w) {
                            y = y * lanes<T>(wi, k);
                        } else if constexpr (with_b) {
                            y = y + lanes<T>(bi, k);
                        }
                        y.put(o + 2 * k);
                    }
                    st_stream<16>(dst + v * 16, pack<T, 16>(o));
                });
            };
            using Yes = std::true_type;
            using No = std::false_type;
            if (SHIFT) {
                write(Yes(), Yes());                 // ones and zeros where there are none
                for (int e = t; e < rv.edges; e += G) {
                    const int j = rv.edge_at(e);
                    const float xh = (ld_elem<T>(in_slot + j) - mean) * rstd;
                    st_elem<T>(p.out, at + rv.edge_col(e),
                               fmaf(xh, ld_elem<T>(ws + j), ld_elem<T>(bs + j)));
                }
            } else if (p.w) {
                if (p.b) write(Yes(), Yes()); else write(Yes(), No());
            } else {
                if (p.b) write(No(), Yes()); else write(No(), No());
            }
        }
        step.next(p.nslots);
    }
    if (n < ring.count) {
        // a wait ran out: report it, and let the copies that are under way land
        if (tid == 0) {
            report_timeout(p.status, kSiteStagedFull);
            ring.drain(step, n);
        }
        __syncthreads();
    }
}

}  // namespace rmsnorm
