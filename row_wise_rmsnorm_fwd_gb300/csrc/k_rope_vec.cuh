// k_rope_vec.cuh -- rotary positions with head norms, heads in vectors.
//
// A head is taken as units of two vectors of EPV elements, half of the turned part apart, so
// that the unit holds EPV whole pairs (interleaved: each vector half of them; vectors of
// one element: neighbours), and behind that half of the rest apart: neighbouring lanes have
// neighbouring vectors, so that no sector of memory is asked for twice.  `lanes` lanes (a
// power of two) share a head, a unit each, so a warp has 32 / lanes heads at a time: of one
// token, or, where a token has fewer, of several.  It walks over its tokens' heads, and its
// lanes keep the cosines and sines of their pairs for all of them: an angle is formed once
// for a warp's share of a token's heads, by one of the lanes that need it.  A CTA works on q
// alone or on k alone, so a lane's weights, and backward its column sums, stay in registers
// for all its tokens.
//
// What bounds it: HBM, where a token has eight rounds of heads or so; with fewer the token's
// position, angles and addresses (about 200 instructions a warp) weigh more, and lanes are
// idle where a head is not a power of two units.  Measured (calls back to back, us and % of
// the HBM copy peak; heads of q + k):
//   forward with norms bf16 65536 tokens, 32 + 8 of 128: 219 (91), interleaved 218 (91), without
//     norms 204 (97); 16 + 16 of 64: 115 (69); 32768, 16 + 4 of 256, 64 turned: 117 (84);
//     fp32 32768, 32 + 8 of 128: 203 (98)
//   backward the same: 316 (94), 320 (93), 204 (97), 162 (73), 166 (89), 310 (96)
//   16 + 16 of 64 without positions (token s stands at s) 103 (77) and 142 (84), without norms too 84 (94)
//     and 84 (94)
//   7 + 1 of 96: 84 (36) and 122 (37); 28 + 4 of 80, 20 turned (vectors of 4 bytes): 373 (27)
//     and 554 (27)
// A warp per head with every angle formed for itself (k_rope.cuh): 1328 and 3876.
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
__device__ __forceinline__ RopeOne minus(RopeOne a, RopeOne b) { return {a.v - b.v}; }
__device__ __forceinline__ Lanes minus(Lanes a, Lanes b) {
    Lanes r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
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

// The lane groups of a token share the work: of NG groups group g (0, 1, ...) forms every NG-th
// pair from g on, and hands it to the others.  first, second: numbers of the two halves of the
// unit's pairs; base: the lane of group 0 that has this lane's unit.
template <int EPV, int NG>
__device__ __forceinline__ void rope_share_angles(RopeAngles<EPV>& t, const uint64_t* freqs, int first,
                                                  int second, int64_t position, float mscale, int lanes,
                                                  int group, int base) {
    constexpr int STEPS = (EPV + NG - 1) / NG;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
        const int k = j * NG + group;
        const int i = k < EPV / 2 || EPV == 1 ? first + k : second + k - EPV / 2;
        const float2 cs = rope_turn(__ldg(freqs + i), position, mscale);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            t.c[j * NG + g] = NG == 1 ? cs.x : __shfl_sync(0xffffffffu, cs.x, base + g * lanes);
            t.s[j * NG + g] = NG == 1 ? cs.y : __shfl_sync(0xffffffffu, cs.y, base + g * lanes);
        }
    }
}

// All lanes of the warp; `share` groups (a power of two) work on the token.
template <int EPV>
__device__ __forceinline__ void rope_angles(RopeAngles<EPV>& t, const uint64_t* freqs, int first, int second,
                                            int64_t position, float mscale, int lanes, int share, int group,
                                            int base) {
    constexpr int N8 = EPV < 8 ? EPV : 8, N4 = EPV < 4 ? EPV : 4, N2 = EPV < 2 ? EPV : 2;
    if (share >= 8) rope_share_angles<EPV, N8>(t, freqs, first, second, position, mscale, lanes, group % N8, base);
    else if (share == 4) rope_share_angles<EPV, N4>(t, freqs, first, second, position, mscale, lanes, group % N4, base);
    else if (share == 2) rope_share_angles<EPV, N2>(t, freqs, first, second, position, mscale, lanes, group % N2, base);
    else rope_share_angles<EPV, 1>(t, freqs, first, second, position, mscale, lanes, 0, base);
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
#pragma unroll
        for (int k = 0; k < RopeVec<EPV>::N; ++k) {
            const L c = L::of(t.c + k * RopeVec<EPV>::PER), s = L::of(t.s + k * RopeVec<EPV>::PER);
            const L x = a.e[k], y = b.e[k];
            if constexpr (BACK) {
                a.e[k] = fma(y, s, x * c);
                b.e[k] = minus(y * c, x * s);
            } else {
                a.e[k] = minus(x * c, y * s);
                b.e[k] = fma(x, s, y * c);
            }
        }
    }
}

// A lane's own vectors of the heads to come, in shared memory: copied there without passing
// through registers, kRopeStages rounds of heads ahead of the one at work and across tokens.
// Nothing is shared among threads, so a thread waits for its own copies and no barrier is
// needed.  Vectors of 2 bytes, which such copies cannot move, are read when their turn comes.
constexpr int kRopeStages = 3;

template <int VB>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, bool yes) {
    const uint32_t n = yes ? VB : 0;            // what is not read is filled with zeros
    if constexpr (VB == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(to), "l"(from), "r"(n) : "memory");
    else if constexpr (VB == 8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" :: "r"(to), "l"(from), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(to), "l"(from), "r"(n) : "memory");
}

template <int VB>
__device__ __forceinline__ Vec<VB> staged_vec(uint32_t at) {
    Vec<VB> v;
    if constexpr (VB == 16)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.u[0]), "=r"(v.u[1]), "=r"(v.u[2]), "=r"(v.u[3]) : "r"(at) : "memory");
    else if constexpr (VB == 8)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.u[0]), "=r"(v.u[1]) : "r"(at) : "memory");
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v.u[0]) : "r"(at) : "memory");
    return v;
}

// CTAs to an SM that the registers have to allow: more of them spill.  Measured (us, bf16
// 65536 tokens, 32 + 8 heads of 128): forward 4 / 5 / 6 CTAs and 4 slots 228 / 230 / 245, 3
// slots and 5 CTAs 224; with the norm's gradient 3 / 4 CTAs 314 / 335, 3 slots 316 / 318.
constexpr int rope_ctas(int kind) { return kind == kRopeGrad ? 3 : 4; }

// LANES > 0: that many lanes to a head, each with a whole unit; 0: p.lanes, of which some may
// have none or half of one.
template <typename T, int VB, bool INTER, int KIND, int LANES>
__global__ void __launch_bounds__(32 * kRopeVecWarps, rope_ctas(KIND)) rope_vec_kernel(const RopeParams p) {
    constexpr int EPV = VecTraits<T, VB>::kElems;
    constexpr bool NEAR = INTER && EPV > 1;
    constexpr bool GRAD = KIND == kRopeGrad, BACK = KIND != kRopeTurn;
    constexpr int VECS = GRAD ? 4 : 2, THREADS = 32 * kRopeVecWarps;
    constexpr bool ASYNC = VB > 2;
    constexpr int STAGE = VECS * THREADS * VB, SUMS = GRAD ? kRopeVecWarps * 64 * EPV * 4 : 0;
    using V = RopeVec<EPV>;
    using L = typename V::L;
    constexpr int STAGED = ASYNC ? kRopeStages * STAGE : 16;
    __shared__ alignas(16) unsigned char smem[STAGED > SUMS ? STAGED : SUMS];
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int which = static_cast<int>(blockIdx.x) >= p.q_ctas;
    const int cta = static_cast<int>(blockIdx.x) - (which ? p.q_ctas : 0);
    const int ctas = which ? static_cast<int>(gridDim.x) - p.q_ctas : p.q_ctas;
    const RopeHeads& t = p.t[which];
    const int lanes = LANES ? LANES : p.lanes;
    const int sub = lane / lanes, l = lane - sub * lanes;
    // the warp's lane groups by token, and the token's groups
    const int share = p.share[which], mine = sub % share, token_of_warp = sub / share;
    const int tokens_per_warp = 32 / lanes / share;
    const int half = p.rot / 2;
    const int turned = half / EPV;                  // units that are turned
    const bool on = LANES || l < p.units, turns = l < turned;
    int ja, jb;                                     // first columns of the two vectors
    if (turns) {
        ja = INTER && !NEAR ? 2 * l : l * EPV;
        jb = INTER && !NEAR ? ja + 1 : ja + half;
    } else {
        ja = p.rot + (l - turned) * EPV;
        jb = ja + (p.units - turned) * EPV;
    }
    const bool on_b = LANES || (on && jb < p.dim);
    // numbers of the two halves of the unit's pairs; lanes that turn nothing take any
    const int unit = turns ? l : 0;
    const int first_pair = NEAR ? unit * EPV / 2 : unit * EPV;
    const int second_pair = first_pair + (NEAR ? half / 2 : EPV / 2);
    const bool all_turn = turned >= lanes;
    auto load = [&](const T* at, bool yes) {
        Vec<VB> v;
        if constexpr (VB == 2) v.h = 0;
        else {
#pragma unroll
            for (int k = 0; k < Vec<VB>::kWords; ++k) v.u[k] = 0u;
        }
        if (yes) v = ld_stream<VB>(at);
        return v;
    };
    pdl_wait();
    Vec<VB> wa, wb;                                 // weights, packed
    const bool weights = t.w != nullptr;
    if (weights) {
        wa = load(static_cast<const T*>(t.w) + ja, on);
        wb = load(static_cast<const T*>(t.w) + jb, on_b);
    }
    V da, db;                                       // column sums
#pragma unroll
    for (int k = 0; k < V::N; ++k) da.e[k] = db.e[k] = L::all(0.f);

    const int heads = t.heads, split = p.split[which];
    const int step = split * share;
    const int ab = jb - ja;
    const RopeView& from = BACK ? t.dy : t.x;
    const int64_t src_step = step * from.head, x_step = GRAD ? step * t.x.head : 0, out_step = step * t.out.head;
    const int64_t items = (p.tokens + tokens_per_warp - 1) / tokens_per_warp * split;
    const int64_t item_step = static_cast<int64_t>(ctas) * kRopeVecWarps;
    const int64_t item0 = static_cast<int64_t>(cta) * kRopeVecWarps + warp;

    // What is read: a round of heads of the warp's tokens at a time.
    struct {
        int64_t item;
        const T *src, *xs;
        int head, rest;              // the lane group's head, and heads from the warp's first on
        bool there;
    } ahead;
    auto enter = [&](int64_t item) {
        ahead.item = item;
        if (item >= items) return;
        const int64_t place = split == 1 ? item : div_nonneg(item, split);
        const int64_t token = place * tokens_per_warp + token_of_warp;
        ahead.there = token < p.tokens;
        const int first = static_cast<int>(item - place * split) * share;
        ahead.head = first + mine;
        ahead.rest = heads - first;
        const int64_t tok = ahead.there ? token : 0, b = div_nonneg(tok, p.seq), s = tok - b * p.seq;
        ahead.src = static_cast<const T*>(from.p) + b * from.batch + s * from.token + ahead.head * from.head + ja;
        if constexpr (GRAD)
            ahead.xs = static_cast<const T*>(t.x.p) + b * t.x.batch + s * t.x.token + ahead.head * t.x.head + ja;
    };
    const uint32_t my_slot = smem_addr(smem) + threadIdx.x * VB;
    auto fetch = [&](int stage) {                    // the next round into `stage`
        if (ahead.item < items) {
            const bool here = ahead.there && ahead.head < heads;
            const uint32_t to = my_slot + stage * STAGE;
            copy_async<VB>(to, ahead.src, here && on);
            copy_async<VB>(to + THREADS * VB, ahead.src + ab, here && on_b);
            ahead.src += src_step;
            if constexpr (GRAD) {
                copy_async<VB>(to + 2 * THREADS * VB, ahead.xs, here && on);
                copy_async<VB>(to + 3 * THREADS * VB, ahead.xs + ab, here && on_b);
                ahead.xs += x_step;
            }
            ahead.head += step;
            ahead.rest -= step;
            if (ahead.rest <= 0) enter(ahead.item + item_step);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    enter(item0);
    if constexpr (ASYNC) {
#pragma unroll
        for (int k = 0; k < kRopeStages - 1; ++k) fetch(k);
    }
    int stage = 0;
    for (int64_t item = item0; item < items; item += item_step) {
        const int64_t place = split == 1 ? item : div_nonneg(item, split);
        const int64_t token = place * tokens_per_warp + token_of_warp;
        const bool there = token < p.tokens;
        const RopeToken tk(p, there ? token : 0);
        const int first = static_cast<int>(item - place * split) * share;
        int head = first + mine;
        T* dst = static_cast<T*>(t.out.p) + tk.at(t.out, head) + ja;
        RopeAngles<EPV> angle;
        rope_angles<EPV>(angle, p.freqs, first_pair, second_pair, tk.position, p.mscale, lanes, share, mine,
                         token_of_warp * share * lanes + l);
        for (int rest = heads - first; rest > 0; rest -= step, head += step) {
            const bool here = there && head < heads;
            struct {
                Vec<VB> a, b, xa, xb;
            } v;
            if constexpr (ASYNC) {
                asm volatile("cp.async.wait_group %0;" :: "n"(kRopeStages - 2) : "memory");
                const uint32_t at = my_slot + stage * STAGE;
                v.a = staged_vec<VB>(at);
                v.b = staged_vec<VB>(at + THREADS * VB);
                if constexpr (GRAD) {
                    v.xa = staged_vec<VB>(at + 2 * THREADS * VB);
                    v.xb = staged_vec<VB>(at + 3 * THREADS * VB);
                }
                // the slot that the round before this one was in
                fetch(stage == 0 ? kRopeStages - 1 : stage - 1);
                stage = stage == kRopeStages - 1 ? 0 : stage + 1;
            } else {
                v.a = load(ahead.src, here && on);
                v.b = load(ahead.src + ab, here && on_b);
                ahead.src += src_step;
                if constexpr (GRAD) {
                    v.xa = load(ahead.xs, here && on);
                    v.xb = load(ahead.xs + ab, here && on_b);
                    ahead.xs += x_step;
                }
                if (rest <= step) enter(item + item_step);
            }
            // widened where they are used: widened once, they would be held so
            if constexpr (VB > 2) {
#pragma unroll
                for (int k = 0; k < Vec<VB>::kWords; ++k) {
                    opaque(wa.u[k]);
                    opaque(wb.u[k]);
                }
            }
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
                    V ua, ub;
                    if (weights) {
                        ua.template widen<T, VB>(wa);
                        ub.template widen<T, VB>(wb);
                    }
#pragma unroll
                    for (int k = 0; k < V::N; ++k) {
                        a.e[k] = a.e[k] * r;
                        b.e[k] = b.e[k] * r;
                        if (weights) {
                            a.e[k] = a.e[k] * ua.e[k];
                            b.e[k] = b.e[k] * ub.e[k];
                        }
                    }
                }
                if (all_turn || turns) rope_apply<EPV, NEAR, BACK>(a, b, angle);
            } else {
                if (all_turn || turns) rope_apply<EPV, NEAR, true>(a, b, angle);
                V x, y, ua, ub;
                x.template widen<T, VB>(v.xa);
                y.template widen<T, VB>(v.xb);
                // what the weights multiply, beside what dw is summed from
                ua = a;
                ub = b;
                if (weights) {
                    V u;
                    u.template widen<T, VB>(wa);
#pragma unroll
                    for (int k = 0; k < V::N; ++k) ua.e[k] = ua.e[k] * u.e[k];
                    u.template widen<T, VB>(wb);
#pragma unroll
                    for (int k = 0; k < V::N; ++k) ub.e[k] = ub.e[k] * u.e[k];
                }
                L s2 = L::all(0.f), s1 = L::all(0.f);
#pragma unroll
                for (int k = 0; k < V::N; ++k) {
                    s2 = fma(y.e[k], y.e[k], fma(x.e[k], x.e[k], s2));
                    s1 = fma(ub.e[k], y.e[k], fma(ua.e[k], x.e[k], s1));
                }
                float ss = group_allreduce_sum(s2.total(), lanes);
                const float dot = group_allreduce_sum(s1.total(), lanes);
                // a head that a lane group lacks: its zeros add nothing, but the factor of
                // zeros is infinite with eps = 0
                if (!here) ss = 1.f;
                const float rstd = rsqrtf(fmaf(ss, p.inv_dim, p.eps));
                const L r = L::all(rstd), less = L::all(-(dot * p.inv_dim * rstd) * rstd);
#pragma unroll
                for (int k = 0; k < V::N; ++k) {
                    da.e[k] = fma(a.e[k], x.e[k] * r, da.e[k]);
                    db.e[k] = fma(b.e[k], y.e[k] * r, db.e[k]);
                    a.e[k] = fma(x.e[k], less, ua.e[k]) * r;
                    b.e[k] = fma(y.e[k], less, ub.e[k]) * r;
                }
            }
            float f[EPV];
            a.put(f);
            if (here && on) st_stream<VB>(dst, pack<T, VB>(f));
            b.put(f);
            if (here && on_b) st_stream<VB>(dst + ab, pack<T, VB>(f));
            dst += out_step;
        }
    }
    if constexpr (GRAD) {
        // the CTA's part: the warp's lane groups, then the warps, in order
        if (!t.dw) return;
        float (*sums)[64 * EPV] = reinterpret_cast<float (*)[64 * EPV]>(smem);
        __syncthreads();                             // every thread is done with its slots
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
