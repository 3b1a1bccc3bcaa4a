// rope_vec_pick.cuh -- instances of the vector kernel of one type and kind.
#pragma once
#include "k_rope_vec.cuh"

namespace rmsnorm {

// Numbers of lanes of their own: heads of 64, 128 and 256 elements in bf16 vectors of 16
// bytes, of 32 to 128 in fp32.  Measured with 4 lanes (us, 65536 tokens, 16 + 16 heads, half layout /
// interleaved, a number of its own first, then one read at run time): bf16 heads of 64 with norms 103,
// 102 / 113, 116, backward 142, 147 / 158, 172, without norms 84, 84 / 85, 87, backward 84, 84 / 85, 85;
// fp32 heads of 32 with norms 84, 84 / 90, 89, backward 132, 122 / 127, 127, without norms 82, 82 / 83, 83,
// backward 93, 92 / 94, 82: the last has none.
template <typename T, int KIND, bool INTER>
static RopeFn rope_pick_vec(int vb, int lanes) {
    if constexpr (sizeof(T) == 2 || KIND != kRopeTurnBack)
        if (vb == 16 && lanes == 4) return rope_vec_kernel<T, 16, INTER, KIND, 4>;
    if (vb == 16 && lanes == 8) return rope_vec_kernel<T, 16, INTER, KIND, 8>;
    if (vb == 16 && lanes == 16) return rope_vec_kernel<T, 16, INTER, KIND, 16>;
    switch (vb) {
        case 16: return rope_vec_kernel<T, 16, INTER, KIND, 0>;
        case 8: return rope_vec_kernel<T, 8, INTER, KIND, 0>;
        case 4: return rope_vec_kernel<T, 4, INTER, KIND, 0>;
        default:
            if constexpr (sizeof(T) == 2) return rope_vec_kernel<T, 2, INTER, KIND, 0>;
            return nullptr;
    }
}

template <typename T, int KIND>
static RopeFn rope_pick_vec_all(int vb, bool interleaved, int lanes) {
    return interleaved ? rope_pick_vec<T, KIND, true>(vb, lanes) : rope_pick_vec<T, KIND, false>(vb, lanes);
}

}  // namespace rmsnorm
