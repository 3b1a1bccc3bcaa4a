// k_rope_vec.cuh -- rotary positions with head norms, heads in vectors.
//
// A head is taken as units of two vectors of EPV elements: where it is turned, the unit
// holds EPV whole pairs (vectors i and i + rot/2, or two neighbours if interleaved), behind
// that two neighbours.  `lanes` lanes (a power of two) share a head, a unit each, so a
// warp has 32 / lanes heads of a token at a time, walks over the token's heads, and its
// lanes keep the cosines and sines of their pairs for all of them: an angle is formed once
// for a warp's share of a token's heads, by one of the lanes that need it.  A CTA works on q alone or on k alone, so a lane's
// weights, and backward its column sums, stay in registers for all its tokens.
#pragma once
#include <type_traits>

#include "k_rope.cuh"
#include "pairs.cuh"

namespace rmsnorm {

// One element, with the operations of a pair (Lanes), for vectors of one element.
struct RopeOne {
    float v;
    static __device__ __forceinline__ RopeOne all(float a) { return {a}; }
    static __device__ __forceinline__ RopeOne of(const float* f) { return {f[0]}; }
    __device__ __forceinline__ RopeOne operator*(RopeOne o) const { return {v * o.v}; }
    __device__ __forceinline__ float total() const { return v; }
    __device__ __forceinline__ void put(float* f) const { f[0] = v; }
};
__device__ __forceinline__ RopeOne fma(RopeOne a, RopeOne b, RopeOne c) { return {fmaf(a.v, b.v, c.v)}; }

// A vector of EPV fp32 elements as pairs.
template <int EPV>
struct RopeVec {
    using L = std::conditional_t<EPV == 1, RopeOne, Lanes>;
    static constexpr int N = EPV == 1 ? 1 : EPV / 2;
    static constexpr int PER = EPV == 1 ? 1 : 2;
    L e[N];
    template <typename T, int VB>
    __device__ __forceinline__ void widen(const Vec<VB>& v) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float f[2];
#pragma unroll
            for (int j = 0; j < PER; ++j) f[j] = get<T, VB>(v, k * PER + j);
            e[k] = L::of(f);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[EPV]) {
#pragma unroll
        for (int k = 0; k < N; ++k) e[k] = L::of(f + k * PER);
    }
    __device__ __forceinline__ void put(float (&f)[EPV]) const {
#pragma unroll
        for (int k = 0; k < N; ++k) e[k].put(f + k * PER);
    }
};

// The cosines and sines of a lane's EPV pairs.  Pair k of a unit belongs to element k of
// both vectors (FAR), or to neighbours: the first half of the pairs in the first vector.
template <int EPV>
struct RopeAngles {
    float c[EPV], s[EPV];
};

// The lane groups of a warp share the work: of NG groups group g forms every NG-th pair from g
// on, and hands it to the others.
template <int EPV, int NG>
__device__ __forceinline__ void rope_share_angles(RopeAngles<EPV>& t, const uint64_t* freqs, int first,
                                                  int second, int64_t position, float mscale, int lanes,
                                                  int sub, int l) {
    constexpr int STEPS = (EPV + NG - 1) / NG;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
        int k = j * NG + sub % NG;
        if (k >= EPV) k = EPV - 1;
        const int i = k < EPV / 2 || EPV == 1 ? first + k : second + k - EPV / 2;
        const float2 cs = rope_turn(__ldg(freqs + i), position, mscale);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (j * NG + g < EPV) {
                t.c[j * NG + g] = NG == 1 ? cs.x : __shfl_sync(0xffffffffu, cs.x, g * lanes + l);
                t.s[j * NG + g] = NG == 1 ? cs.y : __shfl_sync(0xffffffffu, cs.y, g * lanes + l);
            }
        }
    }
}

// All lanes of the warp.  first, second: pair numbers of the two halves of the unit's pairs.
template <int EPV>
__device__ __forceinline__ void rope_angles(RopeAngles<EPV>& t, const uint64_t* freqs, int first, int second,
                                            int64_t position, float mscale, int lanes, int sub, int l) {
    if (lanes <= 4 && EPV >= 8) {
        rope_share_angles<EPV, (EPV < 8 ? EPV : 8)>(t, freqs, first, second, position, mscale, lanes, sub, l);
    } else if (lanes <= 8 && EPV >= 4) {
        rope_share_angles<EPV, (EPV < 4 ? EPV : 4)>(t, freqs, first, second, position, mscale, lanes, sub, l);
    } else if (lanes <= 16 && EPV >= 2) {
        rope_share_angles<EPV, (EPV < 2 ? EPV : 2)>(t, freqs, first, second, position, mscale, lanes, sub, l);
    } else {
        rope_share_angles<EPV, 1>(t, freqs, first, second, position, mscale, lanes, sub, l);
    }
}

// Two vectors turned by their pairs' angles (BACK: the other way).  NEAR: pairs are neighbours.
template <int EPV, bool NEAR, bool BACK>
__device__ __forceinline__ void rope_apply(RopeVec<EPV>& a, RopeVec<EPV>& b, const RopeAngles<EPV>& t) {
    using L = typename RopeVec<EPV>::L;
    if constexpr (NEAR) {
        auto turn = [](L& v, float c, float s) {
            if (BACK) s = -s;
            float f[2], o[2];
            v.put(f);
            o[0] = fmaf(f[0], c, -(f[1] * s));
            o[1] = fmaf(f[1], c, f[0] * s);
            v = L::of(o);
        };
#pragma unroll
        for (int k = 0; k < EPV / 2; ++k) {
            turn(a.e[k], t.c[k], t.s[k]);
            turn(b.e[k], t.c[EPV / 2 + k], t.s[EPV / 2 + k]);
        }
    } else {
        const L minus = L::all(-1.f);
#pragma unroll
        for (int k = 0; k < RopeVec<EPV>::N; ++k) {
            const L c = L::of(t.c + k * RopeVec<EPV>::PER), s = L::of(t.s + k * RopeVec<EPV>::PER);
            const L x = a.e[k], y = b.e[k];
            const L xs = x * s, ys = y * s;
            a.e[k] = fma(x, c, BACK ? ys : ys * minus);
            b.e[k] = fma(y, c, BACK ? xs * minus : xs);
        }
    }
}

// Registers: enough CTAs to an SM for the loads under way to cover HBM's latency.
constexpr int rope_ctas(int kind) { return kind == kRopeGrad ? 4 : 6; }

template <typename T, int VB, bool INTER, int KIND>
__global__ void __launch_bounds__(32 * kRopeVecWarps, rope_ctas(KIND)) rope_vec_kernel(const RopeParams p) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    constexpr bool NEAR = INTER && EPV > 1;
    constexpr bool GRAD = KIND == kRopeGrad, BACK = KIND != kRopeTurn;
    using V = RopeVec<EPV>;
    using L = typename V::L;
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
    // pair numbers of the two halves of the unit's pairs; lanes that turn nothing take any
    const int unit = turns ? l : 0;
    const int first_pair = unit * EPV, second_pair = first_pair + EPV / 2;
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
    V wa, wb;
    if (t.w) {
        wa.template widen<T, VB>(load(t.w, ja, on));
        wb.template widen<T, VB>(load(t.w, jb, on_b));
    } else {
#pragma unroll
        for (int k = 0; k < V::N; ++k) wa.e[k] = wb.e[k] = L::all(1.f);
    }
    V da, db;                                       // column sums
#pragma unroll
    for (int k = 0; k < V::N; ++k) da.e[k] = db.e[k] = L::all(0.f);

    // What a lane reads of a head, the next one under way while one is worked on.
    struct Loads {
        Vec<VB> a, b, xa, xb;
    };
    const int split = p.split[which];
    const int step = split * groups;
    const int64_t items = p.tokens * split;
    for (int64_t item = static_cast<int64_t>(cta) * kRopeVecWarps + warp; item < items;
         item += static_cast<int64_t>(ctas) * kRopeVecWarps) {
        const int64_t token = item / split;
        const RopeToken tk(p, token);
        const RopeView& from = BACK ? t.dy : t.x;
        const T* src = static_cast<const T*>(from.p) + tk.at(from, 0);
        const T* xs = GRAD ? static_cast<const T*>(t.x.p) + tk.at(t.x, 0) : nullptr;
        T* dst = static_cast<T*>(t.out.p) + tk.at(t.out, 0);
        int head = static_cast<int>(item - token * split) * groups + sub;
        auto read = [&](int h) {
            Loads r;
            const bool here = h < t.heads;
            const int64_t at = h * from.head;
            r.a = load(src, at + ja, here && on);
            r.b = load(src, at + jb, here && on_b);
            if constexpr (GRAD) {
                const int64_t ax = h * t.x.head;
                r.xa = load(xs, ax + ja, here && on);
                r.xb = load(xs, ax + jb, here && on_b);
            }
            return r;
        };
        Loads next = read(head);
        RopeAngles<EPV> angle;
        rope_angles<EPV>(angle, p.freqs, first_pair, second_pair, tk.position, p.mscale, lanes, sub, l);
        for (int rest = t.heads - (head - sub); rest > 0; rest -= step, head += step) {
            const Loads v = next;
            const bool here = head < t.heads;
            if (rest > step) next = read(head + step);
            V a, b;
            a.template widen<T, VB>(v.a);
            b.template widen<T, VB>(v.b);
            if constexpr (!GRAD) {
                if (KIND == kRopeTurn && p.norm) {
                    L s = L::all(0.f);
#pragma unroll
                    for (int k = 0; k < V::N; ++k) s = fma(b.e[k], b.e[k], fma(a.e[k], a.e[k], s));
                    const float sum = group_allreduce_sum(s.total(), lanes);
                    const L r = L::all(rsqrtf(fmaf(sum, p.inv_dim, p.eps)));
#pragma unroll
                    for (int k = 0; k < V::N; ++k) {
                        a.e[k] = a.e[k] * r * wa.e[k];
                        b.e[k] = b.e[k] * r * wb.e[k];
                    }
                }
                if (turns) rope_apply<EPV, NEAR, BACK>(a, b, angle);
            } else {
                if (turns) rope_apply<EPV, NEAR, true>(a, b, angle);
                V x, y;
                x.template widen<T, VB>(v.xa);
                y.template widen<T, VB>(v.xb);
                L s2 = L::all(0.f), s1 = L::all(0.f);
#pragma unroll
                for (int k = 0; k < V::N; ++k) {
                    s2 = fma(y.e[k], y.e[k], fma(x.e[k], x.e[k], s2));
                    s1 = fma(b.e[k] * wb.e[k], y.e[k], fma(a.e[k] * wa.e[k], x.e[k], s1));
                }
                float ss = group_allreduce_sum(s2.total(), lanes);
                const float dot = group_allreduce_sum(s1.total(), lanes);
                // a head that a lane group lacks: its zeros add nothing, but the factor of
                // zeros is infinite with eps = 0
                if (!here) ss = 1.f;
                const float rstd = rsqrtf(fmaf(ss, p.inv_dim, p.eps));
                const L r = L::all(rstd), minus = L::all(-(dot * p.inv_dim * rstd) * rstd);
#pragma unroll
                for (int k = 0; k < V::N; ++k) {
                    da.e[k] = fma(a.e[k], x.e[k] * r, da.e[k]);
                    db.e[k] = fma(b.e[k], y.e[k] * r, db.e[k]);
                    a.e[k] = fma(x.e[k], minus, a.e[k] * wa.e[k]) * r;
                    b.e[k] = fma(y.e[k], minus, b.e[k] * wb.e[k]) * r;
                }
            }
            T* to = dst + head * t.out.head;
            float f[EPV];
            a.put(f);
            if (here && on) st_stream<VB>(to + ja, pack<T, VB>(f));
            b.put(f);
            if (here && on_b) st_stream<VB>(to + jb, pack<T, VB>(f));
        }
    }
    if constexpr (GRAD) {
        // the CTA's part: the warp's lane groups, then the warps, in order
        if (!t.dw) return;
        float fa[EPV], fb[EPV];
        da.put(fa);
        db.put(fb);
#pragma unroll
        for (int k = 0; k < EPV; ++k) {
            for (int m = lanes; m < 32; m <<= 1) {
                fa[k] += __shfl_xor_sync(0xffffffffu, fa[k], m);
                fb[k] += __shfl_xor_sync(0xffffffffu, fb[k], m);
            }
            if (sub == 0) {
                if (on) sums[warp][ja + k] = fa[k];
                if (on_b) sums[warp][jb + k] = fb[k];
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
