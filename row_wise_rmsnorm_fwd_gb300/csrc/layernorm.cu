// layernorm.cu -- instances of the layer norm forward kernels, both dtypes.
#include "k_layernorm.cuh"

namespace rmsnorm {

template <typename T>
static NormFn twopass_pick(int vb) {
    switch (vb) {
        case 16: return layernorm_twopass_kernel<T, 16>;
        case 8: return layernorm_twopass_kernel<T, 8>;
        case 4: return layernorm_twopass_kernel<T, 4>;
        case 2:
            if constexpr (sizeof(T) == 2) return layernorm_twopass_kernel<T, 2>;
            return nullptr;
        default: return nullptr;
    }
}

NormFn layernorm_twopass_ptr(int dtype, int vb) {
    return dtype == 0 ? twopass_pick<float>(vb) : twopass_pick<__nv_bfloat16>(vb);
}

NormFn layernorm_staged_ptr(int dtype, bool shift) {
    if (dtype == 0) return shift ? layernorm_staged_kernel<float, true> : layernorm_staged_kernel<float, false>;
    return shift ? layernorm_staged_kernel<__nv_bfloat16, true>
                 : layernorm_staged_kernel<__nv_bfloat16, false>;
}

int layernorm_twopass_block() { return kLayerTwopassThreads; }

}  // namespace rmsnorm
