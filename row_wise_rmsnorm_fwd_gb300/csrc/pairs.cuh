// pairs.cuh -- vectors taken as packed pairs of fp32 elements (the f32x2
// instructions of k_softmax.cuh: two lanes in one issue slot, each rounded as
// the scalar operation), with a scalar stand-in for vectors of one element.
#pragma once
#include "k_softmax.cuh"

namespace rmsnorm {

// A pair, or one element where a vector holds no more: W elements.
template <int W> struct Lanes;
template <> struct Lanes<2> {
    uint64_t v;
    static __device__ __forceinline__ Lanes all(float a) { return {pack_x2(a, a)}; }
    static __device__ __forceinline__ Lanes of(const float* f) { return {pack_x2(f[0], f[1])}; }
    __device__ __forceinline__ float largest(float m) const {
        float a, b;
        unpack_x2(v, a, b);
        return fmaxf(fmaxf(a, b), m);
    }
    __device__ __forceinline__ Lanes operator+(Lanes o) const { return {add_x2(v, o.v)}; }
    __device__ __forceinline__ Lanes operator*(Lanes o) const { return {mul_x2(v, o.v)}; }
    __device__ __forceinline__ float total() const {
        float a, b;
        unpack_x2(v, a, b);
        return a + b;
    }
    __device__ __forceinline__ void put(float* f) const { unpack_x2(v, f[0], f[1]); }
};
template <> struct Lanes<1> {
    float v;
    static __device__ __forceinline__ Lanes all(float a) { return {a}; }
    static __device__ __forceinline__ Lanes of(const float* f) { return {f[0]}; }
    __device__ __forceinline__ float largest(float m) const { return fmaxf(v, m); }
    __device__ __forceinline__ Lanes operator+(Lanes o) const { return {v + o.v}; }
    __device__ __forceinline__ Lanes operator*(Lanes o) const { return {v * o.v}; }
    __device__ __forceinline__ float total() const { return v; }
    __device__ __forceinline__ void put(float* f) const { f[0] = v; }
};

// a * b + c, rounded once.
__device__ __forceinline__ Lanes<2> fma(Lanes<2> a, Lanes<2> b, Lanes<2> c) {
    return {fma_x2(a.v, b.v, c.v)};
}
__device__ __forceinline__ Lanes<1> fma(Lanes<1> a, Lanes<1> b, Lanes<1> c) {
    return {fmaf(a.v, b.v, c.v)};
}

template <typename T, int VB>
struct PairTraits {
    static constexpr int kElems = VecTraits<T, VB>::kElems;
    static constexpr int W = kElems > 1 ? 2 : 1;
    static constexpr int N = kElems / W;
};

// Pair k of a vector, widened exactly to fp32.
template <typename T, int VB>
__device__ __forceinline__ Lanes<PairTraits<T, VB>::W> lanes(const Vec<VB>& v, int k) {
    if constexpr (PairTraits<T, VB>::W == 2) {
        return {pack_x2(get<T, VB>(v, 2 * k), get<T, VB>(v, 2 * k + 1))};
    } else {
        return {get<T, VB>(v, 0)};
    }
}

// Zero the elements from number n (0 <= n) of a vector on.
template <typename T, int VB>
__device__ __forceinline__ void clear_from(Vec<VB>& v, int n) {
    if constexpr (VB == 2) {
        if (n < 1) v.h = 0;
    } else {
        constexpr int PER = 4 / static_cast<int>(sizeof(T));     // elements of a word
#pragma unroll
        for (int k = 0; k < VB / 4; ++k) {
            if (n <= k * PER) v.u[k] = 0u;
            else if (PER == 2 && n == k * PER + 1) v.u[k] &= 0xFFFFu;
        }
    }
}

// Zero the elements below number n (n <= 0: none).
template <typename T, int VB>
__device__ __forceinline__ void clear_below(Vec<VB>& v, int n) {
    constexpr int PER = 4 / static_cast<int>(sizeof(T));
#pragma unroll
    for (int k = 0; k < VB / 4; ++k) {
        if (n >= (k + 1) * PER) v.u[k] = 0u;
        else if (PER == 2 && n == k * PER + 1) v.u[k] &= 0xFFFF0000u;
    }
}

template <int VB>
__device__ __forceinline__ Vec<VB> zero_vec() {
    Vec<VB> v;
    if constexpr (VB == 2) {
        v.h = 0;
    } else {
#pragma unroll
        for (int k = 0; k < VB / 4; ++k) v.u[k] = 0u;
    }
    return v;
}

// A vector of ones.
template <typename T, int VB>
__device__ __forceinline__ Vec<VB> ones_vec() {
    Vec<VB> v;
    if constexpr (VB == 2) {
        v.h = 0x3F80;
    } else {
#pragma unroll
        for (int k = 0; k < VB / 4; ++k) v.u[k] = sizeof(T) == 4 ? 0x3F800000u : 0x3F803F80u;
    }
    return v;
}

// Pair k of a vector plus a pair: for bf16 the mixed-precision addition, which
// widens its operand by itself, one instruction per element where widening and
// a packed addition take one and a half.
template <typename T, int VB>
__device__ __forceinline__ Lanes<PairTraits<T, VB>::W> lanes_plus(
    const Vec<VB>& v, int k, Lanes<PairTraits<T, VB>::W> o) {
    if constexpr (sizeof(T) == 2 && PairTraits<T, VB>::W == 2) {
        float a, b, c, d;
        unpack_x2(o.v, a, b);
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "add.rn.f32.bf16 %0, l, %3;\n\tadd.rn.f32.bf16 %1, h, %4;\n\t}"
            : "=f"(c), "=f"(d) : "r"(v.u[k]), "f"(a), "f"(b));
        return {pack_x2(c, d)};
    } else {
        return lanes<T, VB>(v, k) + o;
    }
}

}  // namespace rmsnorm
