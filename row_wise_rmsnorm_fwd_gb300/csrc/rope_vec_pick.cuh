// rope_vec_pick.cuh -- instances of the vector kernel of one kind.
#pragma once
#include "k_rope_vec.cuh"

namespace rmsnorm {

template <typename T, int KIND, bool INTER>
static RopeFn rope_pick_vec(int vb) {
    switch (vb) {
        case 16: return rope_vec_kernel<T, 16, INTER, KIND>;
        case 8: return rope_vec_kernel<T, 8, INTER, KIND>;
        case 4: return rope_vec_kernel<T, 4, INTER, KIND>;
        default:
            if constexpr (sizeof(T) == 2) return rope_vec_kernel<T, 2, INTER, KIND>;
            return nullptr;
    }
}

template <int KIND>
static RopeFn rope_pick_vec_all(int dtype, int vb, bool interleaved) {
    if (dtype == 0)
        return interleaved ? rope_pick_vec<float, KIND, true>(vb) : rope_pick_vec<float, KIND, false>(vb);
    return interleaved ? rope_pick_vec<__nv_bfloat16, KIND, true>(vb)
                       : rope_pick_vec<__nv_bfloat16, KIND, false>(vb);
}

}  // namespace rmsnorm
