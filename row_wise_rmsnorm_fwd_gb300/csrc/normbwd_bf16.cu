// normbwd_bf16.cu -- instances of the one-pass norm backward kernel, bf16.
#include "k_normbwd.cuh"

namespace rmsnorm {

template <int ELEMS, bool LAYER>
static NormFn pick(int rows, int mode) {
    using T = __nv_bfloat16;
    constexpr int NV = ELEMS / VecTraits<T, 16>::kElems;
    if (rows == 2) {
        if constexpr (ELEMS == 16)
            if (mode == kWhole) return norm_bwd_staged_kernel<T, NV, LAYER, 2, kWhole>;
        if constexpr (ELEMS == 16 && LAYER)
            if (mode == kPartial) return norm_bwd_staged_kernel<T, NV, LAYER, 2, kPartial>;
        return nullptr;
    }
    switch (mode) {
        case kWhole:
            if constexpr (ELEMS == 16 || !LAYER) return norm_bwd_staged_kernel<T, NV, LAYER, 1, kWhole>;
            else return nullptr;
        case kPartial: return norm_bwd_staged_kernel<T, NV, LAYER, 1, kPartial>;
        case kShift: return norm_bwd_staged_kernel<T, NV, LAYER, 1, kShift>;
        default: return nullptr;
    }
}

NormFn norm_bwd_staged_ptr_bf16(int elems, bool layer, int rows, int mode) {
    if (elems == 32) return layer ? pick<32, true>(rows, mode) : pick<32, false>(rows, mode);
    return layer ? pick<16, true>(rows, mode) : pick<16, false>(rows, mode);
}

}  // namespace rmsnorm
