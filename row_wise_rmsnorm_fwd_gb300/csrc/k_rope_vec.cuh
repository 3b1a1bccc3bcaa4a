// k_rope_vec.cuh -- rotary positions with head norms, heads in vectors.
//
// A head is taken as units of two vectors of EPV elements: where it is turned, the unit
// holds EPV whole pairs (vectors i and i + rot/2, or two neighbours if interleaved), behind
// that two neighbours.  `lanes` lanes (a power of two) share a head, a unit each, so a
// warp has 32 / lanes heads of a token at a time, walks over the token's heads, and its
// lanes keep the cosines and sines of their pairs for all of them: an angle is formed once
// for a warp's share of a token's heads.  A CTA works on q alone or on k alone, so a lane's
// weights, and backward its column sums, stay in registers for all its tokens.
#pragma once
#include "k_rope.cuh"

namespace rmsnorm {

template <int EPV>
struct RopeAngles {
    float c[EPV], s[EPV];
};

// Two vectors' elements turned by their pairs' angles (BACK: the other way).  NEAR: the
// pairs are neighbours within a vector, else element k of one and of the other.
template <int EPV, bool NEAR, bool BACK>
__device__ __forceinline__ void rope_apply(float (&a)[EPV], float (&b)[EPV], const RopeAngles<EPV>& t) {
    auto turn = [](float& x, float& y, float c, float s) {
        if (BACK) s = -s;
        const float x0 = x;
        x = fmaf(x0, c, -(y * s));
        y = fmaf(y, c, x0 * s);
    };
    if constexpr (NEAR) {
#pragma unroll
        for (int k = 0; k < EPV / 2; ++k) {
            turn(a[2 * k], a[2 * k + 1], t.c[k], t.s[k]);
            turn(b[2 * k], b[2 * k + 1], t.c[EPV / 2 + k], t.s[EPV / 2 + k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < EPV; ++k) turn(a[k], b[k], t.c[k], t.s[k]);
    }
}

template <typename T, int VB, bool INTER, int KIND>
__global__ void __launch_bounds__(32 * kRopeVecWarps) rope_vec_kernel(const RopeParams p) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    constexpr bool NEAR = INTER && EPV > 1;
    constexpr bool GRAD = KIND == kRopeGrad, BACK = KIND != kRopeTurn;
    constexpr int U = GRAD ? 1 : 2;                 // heads of a lane under way at once
    __shared__ float sums[GRAD ? kRopeVecWarps : 1][GRAD ? 64 * EPV : 1];
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int which = static_cast<int>(blockIdx.x) >= p.q_ctas;
    const int cta = static_cast<int>(blockIdx.x) - (which ? p.q_ctas : 0);
    const int ctas = which ? static_cast<int>(gridDim.x) - p.q_ctas : p.q_ctas;
    const RopeHeads& t = p.t[which];
    const int lanes = p.lanes, groups = 32 / lanes;
    const int sub = lane / lanes, l = lane - sub * lanes;
    const int half = p.rot / 2;
    const int turned = half / EPV;                  // units that are turned
    const bool on = l < p.units, turns = l < turned;
    int ja, jb;                                     // first columns of the two vectors
    if (turns) {
        ja = INTER ? 2 * l * EPV : l * EPV;
        jb = INTER ? ja + EPV : ja + half;
    } else {
        ja = p.rot + 2 * (l - turned) * EPV;
        jb = ja + EPV;
    }
    const bool on_b = on && jb < p.dim;
    auto load = [&](const void* base, int64_t at, bool yes) {
        Vec<VB> v;
        if constexpr (VB == 2) v.h = 0;
        else {
#pragma unroll
            for (int k = 0; k < Vec<VB>::kWords; ++k) v.u[k] = 0u;
        }
        if (yes) v = ld_stream<VB>(static_cast<const T*>(base) + at);
        return v;
    };
    pdl_wait();
    float wa[EPV], wb[EPV];
#pragma unroll
    for (int k = 0; k < EPV; ++k) wa[k] = wb[k] = 1.f;
    if (t.w) {
        const Vec<VB> va = load(t.w, ja, on), vb = load(t.w, jb, on_b);
#pragma unroll
        for (int k = 0; k < EPV; ++k) {
            wa[k] = get<T, VB>(va, k);
            wb[k] = get<T, VB>(vb, k);
        }
    }
    float da[GRAD ? EPV : 1], db[GRAD ? EPV : 1];
#pragma unroll
    for (int k = 0; k < (GRAD ? EPV : 1); ++k) da[k] = db[k] = 0.f;

    const int split = p.split[which];
    const int64_t items = p.tokens * split;
    for (int64_t item = static_cast<int64_t>(cta) * kRopeVecWarps + warp; item < items;
         item += static_cast<int64_t>(ctas) * kRopeVecWarps) {
        const int64_t token = item / split;
        const RopeToken tk(p, token);
        const int64_t xa = tk.at(t.x, 0), oa = tk.at(t.out, 0), ga = BACK ? tk.at(t.dy, 0) : 0;
        RopeAngles<EPV> angle;
#pragma unroll
        for (int k = 0; k < EPV; ++k) {
            angle.c[k] = 1.f;
            angle.s[k] = 0.f;
        }
        if (turns) {
#pragma unroll
            for (int k = 0; k < EPV; ++k) {
                const int i = !INTER ? ja + k : (!NEAR ? l : (k < EPV / 2 ? ja / 2 + k : jb / 2 + k - EPV / 2));
                const float2 cs = rope_turn(__ldg(p.freqs + i), tk.position, p.mscale);
                angle.c[k] = cs.x;
                angle.s[k] = cs.y;
            }
        }
        const int step = split * groups;
        for (int first = static_cast<int>(item - token * split) * groups; first < t.heads; first += U * step) {
            Vec<VB> va[U], vb[U];                   // what is turned
            Vec<VB> xva[GRAD ? U : 1], xvb[GRAD ? U : 1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int head = first + sub + u * step;
                const bool here = head < t.heads;
                const RopeView& v = BACK ? t.dy : t.x;
                const int64_t at = (BACK ? ga : xa) + head * v.head;
                va[u] = load(v.p, at + ja, here && on);
                vb[u] = load(v.p, at + jb, here && on_b);
                if constexpr (GRAD) {
                    const int64_t ax = xa + head * t.x.head;
                    xva[u] = load(t.x.p, ax + ja, here && on);
                    xvb[u] = load(t.x.p, ax + jb, here && on_b);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int head = first + sub + u * step;
                const bool here = head < t.heads;
                float a[EPV], b[EPV];
#pragma unroll
                for (int k = 0; k < EPV; ++k) {
                    a[k] = get<T, VB>(va[u], k);
                    b[k] = get<T, VB>(vb[u], k);
                }
                if constexpr (!GRAD) {
                    if (KIND == kRopeTurn && p.norm) {
                        float s = 0.f;
#pragma unroll
                        for (int k = 0; k < EPV; ++k) s = fmaf(b[k], b[k], fmaf(a[k], a[k], s));
                        const float r = rsqrtf(fmaf(group_allreduce_sum(s, lanes), p.inv_dim, p.eps));
#pragma unroll
                        for (int k = 0; k < EPV; ++k) {
                            a[k] = a[k] * r * wa[k];
                            b[k] = b[k] * r * wb[k];
                        }
                    }
                    if (turns) rope_apply<EPV, NEAR, BACK>(a, b, angle);
                } else {
                    if (turns) rope_apply<EPV, NEAR, true>(a, b, angle);
                    float ss = 0.f, dot = 0.f;
#pragma unroll
                    for (int k = 0; k < EPV; ++k) {
                        const float x = get<T, VB>(xva[u], k), y = get<T, VB>(xvb[u], k);
                        ss = fmaf(y, y, fmaf(x, x, ss));
                        dot = fmaf(b[k] * wb[k], y, fmaf(a[k] * wa[k], x, dot));
                    }
                    ss = group_allreduce_sum(ss, lanes);
                    dot = group_allreduce_sum(dot, lanes);
                    // a head that a lane group lacks: its zeros add nothing, but the factor
                    // of zeros is infinite with eps = 0
                    if (!here) ss = 1.f;
                    const float r = rsqrtf(fmaf(ss, p.inv_dim, p.eps));
                    const float kx = (dot * p.inv_dim * r) * r;
#pragma unroll
                    for (int k = 0; k < EPV; ++k) {
                        const float x = get<T, VB>(xva[u], k), y = get<T, VB>(xvb[u], k);
                        da[k] = fmaf(a[k], x * r, da[k]);
                        db[k] = fmaf(b[k], y * r, db[k]);
                        a[k] = r * fmaf(a[k], wa[k], -(x * kx));
                        b[k] = r * fmaf(b[k], wb[k], -(y * kx));
                    }
                }
                T* out = static_cast<T*>(t.out.p) + oa + head * t.out.head;
                if (here && on) st_stream<VB>(out + ja, pack<T, VB>(a));
                if (here && on_b) st_stream<VB>(out + jb, pack<T, VB>(b));
            }
        }
    }
    if constexpr (GRAD) {
        // the CTA's part: the warp's lane groups, then the warps, in order
        if (!t.dw) return;
#pragma unroll
        for (int k = 0; k < EPV; ++k) {
            for (int m = lanes; m < 32; m <<= 1) {
                da[k] += __shfl_xor_sync(0xffffffffu, da[k], m);
                db[k] += __shfl_xor_sync(0xffffffffu, db[k], m);
            }
            if (sub == 0) {
                if (on) sums[warp][ja + k] = da[k];
                if (on_b) sums[warp][jb + k] = db[k];
            }
        }
        __syncthreads();
        for (int j = threadIdx.x; j < p.dim; j += blockDim.x) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kRopeVecWarps; ++w) v += sums[w][j];
            p.part[static_cast<int64_t>(blockIdx.x) * p.part_stride + j] = v;
        }
    }
}

}  // namespace rmsnorm
