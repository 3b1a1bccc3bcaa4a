// k_rope.cuh -- rotary positions with head norms (formulas in
// include/rmsnorm_rope.h).
//
// Angles.  A frequency is a 64-bit number of turns per position in units of 2^-64:
// the integer product with a position, modulo 2^64, is the angle modulo a turn with
// nothing lost for any position.  Of its upper 32 bits the nearest quarter turn is taken
// away in integers, which leaves at most an eighth of a turn for fp32 to hold: the angle
// is off by three roundings of that (without, of half a turn).
// No fp64, and no table in memory.
#pragma once
#include "common.cuh"
#include "integers.cuh"
#include "rope_launch.h"

namespace rmsnorm {

// (cos, sin) * mscale at a position.  Within an eighth of a turn the Taylor series of sine and
// cosine end at x^9 / 9! and x^10 / 10!: the next terms are below 2^-29 (2^-28 of the sine itself)
// and 2^-33.  In units of 2^-24 both are off by at most 2.4 from the angle (its conversion, the
// constant and their product, each of at most an eighth of a turn, and the turns below 2^-32),
// 1.8 from the series and 1 from mscale.
__device__ __forceinline__ float2 rope_turn(uint64_t freq, int64_t position, float mscale) {
    const uint32_t turns = static_cast<uint32_t>((freq * static_cast<uint64_t>(position)) >> 32);
    const uint32_t quarter = (turns + 0x20000000u) >> 30;
    const float x = static_cast<float>(static_cast<int32_t>(turns - (quarter << 30))) *
                    1.4629180792671596e-9f;                        // 2 pi / 2^32
    const float q = x * x;
    float s = fmaf(q, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(q, s, 1.f / 120.f);
    s = fmaf(q, s, -1.f / 6.f);
    s = fmaf(x * q, s, x);
    float c = fmaf(q, -1.f / 3628800.f, 1.f / 40320.f);
    c = fmaf(q, c, -1.f / 720.f);
    c = fmaf(q, c, 1.f / 24.f);
    c = fmaf(q, c, -0.5f);
    c = fmaf(q, c, 1.f);
    const float a = quarter & 1 ? -s : c, b = quarter & 1 ? c : s;
    const float scale = quarter & 2 ? -mscale : mscale;
    return make_float2(a * scale, b * scale);
}

// Position of a token, and where it lies in a view.
struct RopeToken {
    int64_t b, s, position;
    __device__ __forceinline__ RopeToken(const RopeParams& p, int64_t token) {
        b = div_nonneg(token, p.seq);
        s = token - b * p.seq;
        position = p.start;
        if (!p.positions) {
            position += s;
        } else {
            const int64_t n = p.n_positions;
            const int64_t at = token < n ? token : n == p.seq ? s : token % n;
            position += p.wide ? static_cast<const int64_t*>(p.positions)[at]
                               : static_cast<const int32_t*>(p.positions)[at];
        }
    }
    __device__ __forceinline__ int64_t at(const RopeView& v, int64_t head) const {
        return b * v.batch + s * v.token + head * v.head;
    }
};

template <typename T>
__device__ __forceinline__ float rope_elem(const void* p, int64_t at) {
    return static_cast<float>(static_cast<const T*>(p)[at]);
}
template <typename T>
__device__ __forceinline__ void rope_put(void* p, int64_t at, float v) {
    static_cast<T*>(p)[at] = static_cast<T>(v);      // to nearest even
}

// Any head_dim, strides and alignment: a warp per head, which reads it twice, element
// by element, and forms every angle for itself (about thirty instructions each: they
// bound it).  Lane l has the pairs, and behind rot the elements, l, l + 32, ...; both
// elements of a pair are read before either is written, so the heads may be turned in
// place.  BACK: turned the other way, then the norm's gradient; a lane's columns are
// the same for every head, so each warp keeps its own column sums in shared memory.
template <typename T, bool INTER, bool BACK>
__global__ void __launch_bounds__(32 * kRopeAnyWarps) rope_any_kernel(const RopeParams p) {
    __shared__ float sums[BACK ? kRopeAnyWarps : 1][BACK ? 2 * kRopeMaxDim : 1];
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = p.rot / 2;
    if constexpr (BACK) {
        for (int j = lane; j < 2 * p.dim; j += 32) sums[warp][j] = 0.f;
        __syncwarp();
    }
    pdl_wait();
    const int heads = p.t[0].heads + p.t[1].heads;
    const int64_t items = p.tokens * heads;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeAnyWarps + warp; item < items;
         item += static_cast<int64_t>(gridDim.x) * kRopeAnyWarps) {
        const int64_t token = item / heads;
        int head = static_cast<int>(item - token * heads);
        const int which = head >= p.t[0].heads;
        if (which) head -= p.t[0].heads;
        const RopeHeads& t = p.t[which];
        const RopeToken tk(p, token);
        const int64_t xa = tk.at(t.x, head), oa = tk.at(t.out, head);
        const int64_t da = BACK ? tk.at(t.dy, head) : 0;
        auto weight = [&](int j) { return t.w ? rope_elem<T>(t.w, j) : 1.f; };
        // the pair's columns, or a column behind rot twice
        auto columns = [&](int i, int& j0, int& j1) {
            if (i < half) {
                j0 = INTER ? 2 * i : i;
                j1 = INTER ? 2 * i + 1 : i + half;
            } else {
                j0 = j1 = i + half;
            }
        };
        const int units = p.dim - half;             // pairs, then single elements
        if constexpr (!BACK) {
            float r = 1.f;
            if (p.norm) {
                float s = 0.f;
                for (int j = lane; j < p.dim; j += 32) {
                    const float v = rope_elem<T>(t.x.p, xa + j);
                    s = fmaf(v, v, s);
                }
                r = rsqrtf(fmaf(warp_allreduce_sum(s), p.inv_dim, p.eps));
            }
            for (int i = lane; i < units; i += 32) {
                int j0, j1;
                columns(i, j0, j1);
                float a = rope_elem<T>(t.x.p, xa + j0), b = rope_elem<T>(t.x.p, xa + j1);
                if (p.norm) {
                    a = a * r * weight(j0);
                    b = b * r * weight(j1);
                }
                if (i < half) {
                    const float2 cs = rope_turn(p.freqs[i], tk.position, p.mscale);
                    rope_put<T>(t.out.p, oa + j0, fmaf(a, cs.x, -(b * cs.y)));
                    rope_put<T>(t.out.p, oa + j1, fmaf(b, cs.x, a * cs.y));
                } else {
                    rope_put<T>(t.out.p, oa + j0, a);
                }
            }
        } else {
            auto turned = [&](int i, int j0, int j1, float& a, float& b) {
                a = rope_elem<T>(t.dy.p, da + j0);
                b = rope_elem<T>(t.dy.p, da + j1);
                if (i < half) {
                    const float2 cs = rope_turn(p.freqs[i], tk.position, p.mscale);
                    const float a0 = a;
                    a = fmaf(a0, cs.x, b * cs.y);
                    b = fmaf(b, cs.x, -(a0 * cs.y));
                }
            };
            float r = 1.f, k = 0.f;
            if (p.norm) {
                float ss = 0.f, dot = 0.f;
                for (int i = lane; i < units; i += 32) {
                    int j0, j1;
                    columns(i, j0, j1);
                    float a, b;
                    turned(i, j0, j1, a, b);
                    const float x0 = rope_elem<T>(t.x.p, xa + j0);
                    ss = fmaf(x0, x0, ss);
                    dot = fmaf(a * weight(j0), x0, dot);
                    if (i < half) {
                        const float x1 = rope_elem<T>(t.x.p, xa + j1);
                        ss = fmaf(x1, x1, ss);
                        dot = fmaf(b * weight(j1), x1, dot);
                    }
                }
                r = rsqrtf(fmaf(warp_allreduce_sum(ss), p.inv_dim, p.eps));
                k = (warp_allreduce_sum(dot) * p.inv_dim * r) * r;
            }
            for (int i = lane; i < units; i += 32) {
                int j0, j1;
                columns(i, j0, j1);
                float a, b;
                turned(i, j0, j1, a, b);
                if (p.norm) {
                    float* sum = sums[warp] + which * p.dim;
                    const float x0 = rope_elem<T>(t.x.p, xa + j0);
                    const float x1 = rope_elem<T>(t.x.p, xa + j1);
                    sum[j0] = fmaf(a, x0 * r, sum[j0]);
                    a = r * fmaf(a, weight(j0), -(x0 * k));
                    if (i < half) {
                        sum[j1] = fmaf(b, x1 * r, sum[j1]);
                        b = r * fmaf(b, weight(j1), -(x1 * k));
                    }
                }
                rope_put<T>(t.out.p, oa + j0, a);
                if (i < half) rope_put<T>(t.out.p, oa + j1, b);
            }
        }
    }
    if constexpr (BACK) {
        if (!p.part) return;
        __syncthreads();
        for (int j = threadIdx.x; j < 2 * p.dim; j += blockDim.x) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kRopeAnyWarps; ++w) v += sums[w][j];
            p.part[static_cast<int64_t>(blockIdx.x) * p.part_stride + j] = v;
        }
    }
}

// dw from the parts: 32 columns a CTA, each warp every 32nd part, then the warps in order.
static __global__ void __launch_bounds__(kRopeReduceThreads) rope_reduce_kernel(const RopeParams p) {
    constexpr int WARPS = kRopeReduceThreads / 32;
    __shared__ float red[WARPS][33];
    pdl_trigger();
    pdl_wait();
    const RopeHeads& t = p.t[blockIdx.y];
    if (!t.dw) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * 32 + lane;
    const float* from = p.part + p.part_at[blockIdx.y] + (col < p.dim ? col : 0);
    const int n = p.part_n[blockIdx.y];
    float s = 0.f;
    for (int k = warp; k < n; k += WARPS) s += from[static_cast<int64_t>(k) * p.part_stride];
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < p.dim) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += red[w][lane];
        t.dw[col] = v;
    }
}

}  // namespace rmsnorm
