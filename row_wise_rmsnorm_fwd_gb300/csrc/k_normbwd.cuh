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
#include "k_blockring.cuh"
#include "norm_launch.h"
#include "pairs.cuh"

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

// ------------------------------------------------- rows staged: one pass --
// x and dy are read from HBM once: blocks of R * p.rows_per_cta rows come into
// shared memory by bulk copies (k_blockring.cuh); G threads work on R rows at a
// time, NV vectors per thread and row.  Each iteration forms the rows' two
// sums, has one block barrier, and then reads the slot again for dx.  The
// column sums stay in registers (a thread has the same columns of every row it
// sees) until the CTA's rows are done; its row groups are then added through
// shared memory and written as one part.
//
// At 6 bytes an element (bf16) the issue slots are as scarce as the bandwidth,
// so the arithmetic is on packed pairs and arranged for few operations: with
// u = x - mean (RMSNorm: x), the first pass needs d * u once for both
// m(g * xh) and dw, and dx = (d * w + k1 + u * k2) * rstd with two constants of
// the row, k1 = -m(g) and k2 = -m(g * xh) * rstd (which times rstd once more, for
// rows whose squares are near fp32's smallest numbers, would overflow, though dx
// does not).  R = 2 gives each thread two independent rows between barriers.
// Modes: kWhole: every thread has NV whole vectors and there are weights;
// kPartial: aligned rows of any length, with or without weights; kShift: rows
// of any length, the weights copied to shared memory in their layout, a
// shifted row's edges taken by one thread per element.  Vectors past the row's
// end are read as zeros: they add nothing anywhere and are not stored.
//
// Rows of more than 512 threads of 16 elements take 32 per thread (all of a
// thread's 128 registers) rather than the kernels above, which read them twice.
// Layer norm's then take kPartial also where they fill their threads: its weights
// under a predicate are not kept from pass to pass in registers that it lacks
// (kWhole / kPartial: fp32 8192 x 12288 242 / 206 us, bf16 16384 x 16384 314 / 276).
//
// Measured (calls back to back, % of the HBM copy peak): layer norm bf16 65536 x 8192
// 531 us, 89, 16384 x 16384 276 us, 86; fp32 32768 x 4096 241 us, 98; RMSNorm bf16
// 65536 x 4096 243 us, 98, 65536 x 8192 493 us, 96, 16384 x 16384 238 us, 100.  What
// is left in bf16 layer norm is the trips to shared memory (an access per vector
// and pass, waited for by a quarter of the SM's warps: 127 registers each).  Rows
// of any length: bf16 16384 x 4097 117 us, 51.  The three kernels above instead:
// 910 us for bf16 65536 x 8192, 469 us for fp32 32768 x 4096.
enum : int { kWhole, kPartial, kShift };

// Registers per thread, at most: RMSNorm with one row of 16 elements between
// barriers wants resident warps more than registers.  Measured (us, at most 64 /
// 80 / 96 / 128): RMSNorm bf16 shifted 16384 x 4097 106 / 99 / 104 / -; layer norm
// bf16 shifted 16384 x 4097 - / 178 / 123 / 114, 8191 x 2050 - / 60 / 40 / 38.
constexpr int norm_bwd_regs(int elems, bool layer, int rows) {
    return elems == 32 || rows == 2 || layer ? 128 : 80;
}

// v += W floats at `from` (W = 4: on a 16-byte boundary).
template <int W>
__device__ __forceinline__ void add_row(float (&v)[W], const float* from) {
    if constexpr (W == 4) {
        const float4 f = *reinterpret_cast<const float4*>(from);
        v[0] += f.x;
        v[1] += f.y;
        v[2] += f.z;
        v[3] += f.w;
    } else {
        v[0] += *from;
    }
}

template <typename T, int NV, bool LAYER, int R, int MODE>
__global__ void
__maxnreg__((norm_bwd_regs(NV * VecTraits<T, 16>::kElems, LAYER, R)))
norm_bwd_staged_kernel(const NormParams p) {
    constexpr int EPV = VecTraits<T, 16>::kElems;
    constexpr int PN = kPairs<T>;
    constexpr bool SHIFT = MODE == kShift;
    // 32 elements per thread are for rows of more than 8192: a CTA's block is one row, and
    // with threads rounded up to a warp only a thread's last vector may be missing
    constexpr bool WIDE = NV * EPV > 16;
    using L = Lanes;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ alignas(8) uint64_t bars[kBlockRingMaxSlots];
    __shared__ float2 red[2][R][32];
    pdl_trigger();
    const int G = p.group;
    const int width = G < 32 ? G : 32;
    const int tid = threadIdx.x;
    const int g = tid / G;
    const int t = tid - g * G;
    const int warp = tid >> 5, lane = tid & 31;
    const int wpg = G >> 5;
    const int gw0 = g * wpg;
    const int rpc = p.rows_per_cta;          // row groups of the CTA

    const RowRing<T, SHIFT, 2> ring(p, R * rpc, smem, bars);
    const RowVecs<T, SHIFT> rv(ring.shift, p.hidden);
    int merge_width = 1;
    while (merge_width < wpg) merge_width <<= 1;
    bool valid[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        valid[i] = MODE == kWhole || (WIDE && i < NV - 1) || i * G + t < rv.nvec;
    __syncthreads();
    pdl_wait();
    if (warp == 0) ring.prologue();

    const char* wg = static_cast<const char*>(p.w) + t * 16;
    uint32_t ws = 0;
    if constexpr (SHIFT) {
        T* wc = reinterpret_cast<T*>(smem + (ring.base(p.nslots, 0) - ring.base(0, 0)));
        copy_shifted<T>(wc, p.w, rv.skip, p.hidden, ring.row_slot() / static_cast<int>(sizeof(T)), 1.f);
        ws = smem_addr(wc);
        __syncthreads();
    }
    // this thread's edge element (there are at most 14 and G >= 16), its weight and sums
    const bool edge = SHIFT && t < rv.edges;
    const int edge_at = edge ? rv.edge_at(t) : 0;
    const float edge_w = edge ? ld_elem<T>(ws + edge_at) : 0.f;
    float edge_aw = 0.f, edge_ab = 0.f;
    ws += rv.vec_at() + t * 16;
    L aw[NV * PN], ab[LAYER ? NV * PN : 1];
#pragma unroll
    for (int k = 0; k < NV * PN; ++k) aw[k] = L::all(0.f);
#pragma unroll
    for (int k = 0; k < (LAYER ? NV * PN : 1); ++k) ab[k] = L::all(0.f);
    // row r of the group's R rows of this block: row + r * apart
    const int apart = rpc * ring.period();
    int64_t row = ring.first + static_cast<int64_t>(g) * ring.period();
    float mean[R], rstd[R];
    auto stats = [&](int64_t from, float (&m)[R], float (&q)[R]) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = q[r] = 0.f;
            if (LAYER && from + r * apart < p.rows) {
                m[r] = p.mean[from + r * apart];
                q[r] = p.rstd[from + r * apart];
            }
        }
    };
    stats(row, mean, rstd);
    // Whether row r of the block is one of the rows: the last block may lack some.
    // Their vectors are read as zeros and add nothing, but RMSNorm's rstd of zeros is
    // infinite with eps = 0 and would make dw NaN: they take a sum of squares of 1, or,
    // in fp32 with one row between barriers, whose registers that spills, skip the second
    // pass.  Measured (us, sum of 1 / skip): fp32 65536 x 768 115 / 108, 32768 x 4096
    // (two rows) 248 / 250, bf16 65536 x 1280 96 / 99.
    constexpr bool SKIP = !LAYER && sizeof(T) == 4 && R == 1;
    auto in_range = [&](int r) { return WIDE || row + r * apart < p.rows; };
    auto weights = [&](int i) {
        if constexpr (SHIFT) return ld_slot_if(ws + i * G * 16, valid[i]);
        else if constexpr (MODE == kWhole) return ld_ro<16>(wg + i * G * 16);
        else return p.w && valid[i] ? ld_ro<16>(wg + i * G * 16) : ones_vec<T>();
    };
    RingStep step;
    int n = 0;
    for (; n < ring.count; ++n, row += ring.step) {
        // the next rows' statistics, under way while this block is awaited
        float next_mean[R], next_rstd[R];
        stats(row + ring.step, next_mean, next_rstd);
        const bool ok = ring.wait(step);
        ring.finish(step.slot, n);
        const uint32_t in_slot = static_cast<uint32_t>(g * ring.row_slot() + rv.vec_at() + t * 16);
        const uint32_t xs = ring.base(step.slot, 0) + in_slot;
        const uint32_t ds = ring.base(step.slot, 1) + in_slot;
        const uint32_t edge_x = ring.base(step.slot, 0) + static_cast<uint32_t>(g * ring.row_slot() + edge_at);
        const uint32_t edge_d = ring.base(step.slot, 1) + static_cast<uint32_t>(g * ring.row_slot() + edge_at);
        const uint32_t next_row = static_cast<uint32_t>(rpc * ring.row_slot());

        float a[R], b[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool here = in_range(r);
            const L minus = L::all(-mean[r]), q = L::all(rstd[r]);
            L sa = L::all(0.f), sb = L::all(0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const bool on = here && valid[i];
                const Vec<16> x = ld_slot_if(xs + r * next_row + i * G * 16, on);
                const Vec<16> d = ld_slot_if(ds + r * next_row + i * G * 16, on);
                const Vec<16> w = weights(i);
#pragma unroll
                for (int k = 0; k < PN; ++k) {
                    const L dk = lanes<T>(d, k), wk = lanes<T>(w, k);
                    L u;
                    if constexpr (LAYER) u = lanes_plus<T>(x, k, minus);
                    else u = lanes<T>(x, k);
                    const L du = dk * u;
                    if constexpr (LAYER) {
                        sa = fma(dk, wk, sa);
                        aw[i * PN + k] = fma(du, q, aw[i * PN + k]);
                        ab[i * PN + k] = ab[i * PN + k] + dk;
                    } else {
                        sa = fma(u, u, sa);
                    }
                    sb = fma(du, wk, sb);
                }
            }
            a[r] = LAYER || SKIP || here ? sa.total() : 1.f;
            b[r] = sb.total();
            if (SHIFT && edge && here) {
                const float d = ld_elem<T>(edge_d), u = ld_elem<T>(edge_x) - mean[r];
                a[r] = LAYER ? fmaf(d, edge_w, a[r]) : fmaf(u, u, a[r]);
                b[r] = fmaf(d * u, edge_w, b[r]);
                if (LAYER) {
                    edge_aw = fmaf(d * u, rstd[r], edge_aw);
                    edge_ab += d;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            a[r] = share_sum(a[r], width);
            b[r] = share_sum(b[r], width);
        }
        if (wpg > 1 && lane == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) red[n & 1][r][warp] = make_float2(a[r], b[r]);
        }
        if (__syncthreads_or(!ok)) break;            // uniform; also frees the previous slot
        if (warp == 0) ring.refill(step, n);
        if (wpg > 1) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float2 e = make_float2(0.f, 0.f);
                if (lane < wpg) e = red[n & 1][r][gw0 + lane];
                a[r] = group_allreduce_sum(e.x, merge_width);
                b[r] = group_allreduce_sum(e.y, merge_width);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                a[r] = __shfl_sync(0xffffffffu, a[r], 0);
                b[r] = __shfl_sync(0xffffffffu, b[r], 0);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool here = in_range(r);
            if (SKIP && !here) continue;
            float k1 = 0.f;
            if constexpr (LAYER) {
                k1 = -a[r] * p.inv_hidden;
            } else {
                rstd[r] = rsqrtf(fmaf(a[r], p.inv_hidden, p.eps));
            }
            // u * k2 = -xh * m(g * xh), m(g * xh) = rstd * b / H
            const float k2 = -(b[r] * p.inv_hidden * rstd[r]) * rstd[r];
            const L minus = L::all(-mean[r]), q = L::all(rstd[r]);
            const L c1 = L::all(k1), c2 = L::all(k2);
            const int64_t at = (row + r * apart) * p.hidden;
            char* dst = static_cast<char*>(p.out) + (at + rv.head) * static_cast<int>(sizeof(T)) + t * 16;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const bool on = here && valid[i];
                const Vec<16> x = ld_slot_if(xs + r * next_row + i * G * 16, on);
                const Vec<16> d = ld_slot_if(ds + r * next_row + i * G * 16, on);
                const Vec<16> w = weights(i);
                float o[EPV];
#pragma unroll
                for (int k = 0; k < PN; ++k) {
                    const L dk = lanes<T>(d, k), wk = lanes<T>(w, k);
                    if constexpr (LAYER) {
                        const L u = lanes_plus<T>(x, k, minus);
                        (fma(u, c2, fma(dk, wk, c1)) * q).put(o + 2 * k);
                    } else if constexpr (WIDE) {
                        const L u = lanes<T>(x, k);
                        aw[i * PN + k] = fma(dk * u, q, aw[i * PN + k]);
                        (fma(u, c2, dk * wk) * q).put(o + 2 * k);
                    } else {        // as many operations in another order: 3% less time here,
                                    // 4% more in rows of more than 8192 elements
                        const L xh = lanes<T>(x, k) * q;
                        aw[i * PN + k] = fma(dk, xh, aw[i * PN + k]);
                        fma(xh, c2, dk * wk * q).put(o + 2 * k);
                    }
                }
                if (on) st_stream<16>(dst + i * G * 16, pack<T, 16>(o));
            }
            if (SHIFT && edge && here) {
                const float d = ld_elem<T>(edge_d), u = ld_elem<T>(edge_x) - mean[r];
                if (!LAYER) edge_aw = fmaf(d * u, rstd[r], edge_aw);
                st_elem<T>(p.out, at + rv.edge_col(t), rstd[r] * fmaf(u, k2, fmaf(d, edge_w, k1)));
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] = next_mean[r];
            rstd[r] = next_rstd[r];
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
        return;
    }
    // The CTA's part.  One row group: straight from the registers; more: their sums,
    // in order, through shared memory (whose ring is done with and has room for
    // both arrays), as do shifted rows, whose vectors are not on boundaries here.
    auto put_vectors = [&](const L* acc, float* to) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!valid[i]) continue;
            float* at = to + rv.col(i * G + t);
            float f[EPV];
#pragma unroll
            for (int k = 0; k < PN; ++k) acc[i * PN + k].put(f + 2 * k);
#pragma unroll
            for (int k = 0; k < EPV; k += SHIFT ? 1 : 4) {
                if constexpr (SHIFT) at[k] = f[k];
                else *reinterpret_cast<float4*>(at + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
            }
        }
    };
    const int64_t mine = static_cast<int64_t>(blockIdx.x) * p.hidden;
    if (!SHIFT && rpc == 1) {
        if (p.part_w) put_vectors(aw, p.part_w + mine);
        if (LAYER && p.part_b) put_vectors(ab, p.part_b + mine);
        return;
    }
    if (!p.part_w && !p.part_b) return;
    float* sums_w = reinterpret_cast<float*>(smem);
    float* sums_b = sums_w + rpc * p.hidden;
    __syncthreads();
    put_vectors(aw, sums_w + g * p.hidden);
    if (LAYER) put_vectors(ab, sums_b + g * p.hidden);
    if (edge) {
        sums_w[g * p.hidden + rv.edge_col(t)] = edge_aw;
        if (LAYER) sums_b[g * p.hidden + rv.edge_col(t)] = edge_ab;
    }
    __syncthreads();
    auto write_part = [&](const float* sums, float* part) {
        constexpr int W = SHIFT ? 1 : 4;
        for (int c = tid * W; c < p.hidden; c += blockDim.x * W) {
            float v[W];
#pragma unroll
            for (int k = 0; k < W; ++k) v[k] = 0.f;
            for (int r = 0; r < rpc; ++r) add_row<W>(v, sums + r * p.hidden + c);
            if constexpr (W == 1) part[mine + c] = v[0];
            else *reinterpret_cast<float4*>(part + mine + c) = make_float4(v[0], v[1], v[2], v[3]);
        }
    };
    if (p.part_w) write_part(sums_w, p.part_w);
    if (LAYER && p.part_b) write_part(sums_b, p.part_b);
}

// dw and db from the parts, W columns per thread (4 where the columns are a
// multiple of 4: 16-byte loads): a CTA takes 8 * W columns, of which each of its
// 32 lanes adds every 32nd part, ten loads in flight, then the lanes in order.
// grid.y: 0 = dw, 1 = db.  Measured, with the writing of the parts: 3.3 of 21.9 us
// (fp32 2048 x 3584, 304 parts; through shared memory and with 4-byte loads 7.7).
template <int W>
static __global__ void __launch_bounds__(kNormReduceThreads)
norm_bwd_reduce_kernel(const NormParams p) {
    constexpr int COLS = kNormReduceCols, LANES = kNormReduceThreads / COLS;
    __shared__ float red[kNormReduceThreads / 32][COLS * W];
    pdl_trigger();
    pdl_wait();
    const int c = threadIdx.x % COLS, l = threadIdx.x / COLS;
    const int64_t col = (static_cast<int64_t>(blockIdx.x) * COLS + c) * W;
    const float* part = blockIdx.y ? p.part_b : p.part_w;
    float* out = blockIdx.y ? p.db : p.dw;
    if (!part) return;
    // loads past the last part repeat it and are not added
    constexpr int U = 10;
    const float* from = part + (col < p.hidden ? col : 0);
    float s[W];
#pragma unroll
    for (int w = 0; w < W; ++w) s[w] = 0.f;
    for (int k = l; k < p.parts; k += U * LANES) {
        float v[U][W];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int w = 0; w < W; ++w) v[u][w] = 0.f;
            add_row<W>(v[u], from + static_cast<int64_t>(min(k + u * LANES, p.parts - 1)) * p.hidden);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k + u * LANES < p.parts) {
#pragma unroll
                for (int w = 0; w < W; ++w) s[w] += v[u][w];
            }
        }
    }
    // the warp's lanes, then the warps
#pragma unroll
    for (int w = 0; w < W; ++w) {
#pragma unroll
        for (int m = COLS; m < 32; m <<= 1) s[w] += __shfl_xor_sync(0xffffffffu, s[w], m);
        if ((threadIdx.x & 31) < COLS) red[threadIdx.x >> 5][c * W + w] = s[w];
    }
    __syncthreads();
    const int64_t mine = static_cast<int64_t>(blockIdx.x) * COLS * W + threadIdx.x;
    if (threadIdx.x < COLS * W && mine < p.hidden) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kNormReduceThreads / 32; ++k) v += red[k][threadIdx.x];
        out[mine] = v;
    }
}

}  // namespace rmsnorm
