// pairs.cuh -- 16-byte vectors taken as packed pairs of fp32 elements (the f32x2
// instructions of k_softmax.cuh: two lanes in one issue slot, each rounded as
// the scalar operation).
#pragma once
#include "k_softmax.cuh"

namespace rmsnorm {

// A pair of elements.
struct Lanes {
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

// a * b + c, rounded once.
__device__ __forceinline__ Lanes fma(Lanes a, Lanes b, Lanes c) {
    return {fma_x2(a.v, b.v, c.v)};
}

// Pairs of a vector.
template <typename T>
constexpr int kPairs = VecTraits<T, 16>::kElems / 2;

// Pair k of a vector, widened exactly to fp32.
template <typename T>
__device__ __forceinline__ Lanes lanes(const Vec<16>& v, int k) {
    return {pack_x2(get<T, 16>(v, 2 * k), get<T, 16>(v, 2 * k + 1))};
}

// Zero the elements from number n (0 <= n) of a vector on.
template <typename T>
__device__ __forceinline__ void clear_from(Vec<16>& v, int n) {
    constexpr int PER = 4 / static_cast<int>(sizeof(T));     // elements of a word
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (n <= k * PER) v.u[k] = 0u;
        else if (PER == 2 && n == k * PER + 1) v.u[k] &= 0xFFFFu;
    }
}

// Zero the elements below number n (n <= 0: none).
template <typename T>
__device__ __forceinline__ void clear_below(Vec<16>& v, int n) {
    constexpr int PER = 4 / static_cast<int>(sizeof(T));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (n >= (k + 1) * PER) v.u[k] = 0u;
        else if (PER == 2 && n == k * PER + 1) v.u[k] &= 0xFFFF0000u;
    }
}

// A vector of one word over and over: zeros, or ones.
__device__ __forceinline__ Vec<16> words_vec(uint32_t w) {
    Vec<16> v;
#pragma unroll
    for (int k = 0; k < 4; ++k) v.u[k] = w;
    return v;
}
__device__ __forceinline__ Vec<16> zero_vec() { return words_vec(0u); }
template <typename T>
__device__ __forceinline__ Vec<16> ones_vec() {
    return words_vec(sizeof(T) == 4 ? 0x3F800000u : 0x3F803F80u);
}

// Pair k of a vector plus a pair: for bf16 the mixed-precision addition, which
// widens its operand by itself, one instruction per element where widening and
// a packed addition take one and a half.
template <typename T>
__device__ __forceinline__ Lanes lanes_plus(const Vec<16>& v, int k, Lanes o) {
    if constexpr (sizeof(T) == 2) {
        float a, b, c, d;
        unpack_x2(o.v, a, b);
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "add.rn.f32.bf16 %0, l, %3;\n\tadd.rn.f32.bf16 %1, h, %4;\n\t}"
            : "=f"(c), "=f"(d) : "r"(v.u[k]), "f"(a), "f"(b));
        return {pack_x2(c, d)};
    } else {
        return lanes<T>(v, k) + o;
    }
}

}  // namespace rmsnorm
