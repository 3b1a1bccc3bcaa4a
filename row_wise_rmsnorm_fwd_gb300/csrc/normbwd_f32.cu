// normbwd_f32.cu -- instances of the one-pass norm backward kernel, fp32.
#include "k_normbwd.cuh"

namespace rmsnorm {

template <int VB, bool LAYER>
static NormFn pick(int rows, bool full) {
    using T = float;
    constexpr int NV = kNormBwdElems / VecTraits<T, VB>::kElems;
    if (!full) return rows == 1 ? norm_bwd_staged_kernel<T, VB, NV, LAYER, 1, false> : nullptr;
    return rows == 1 ? norm_bwd_staged_kernel<T, VB, NV, LAYER, 1, true>
                     : norm_bwd_staged_kernel<T, VB, NV, LAYER, 2, true>;
}

template <int VB>
static NormFn staged(bool layer, int rows, bool full) {
    return layer ? pick<VB, true>(rows, full) : pick<VB, false>(rows, full);
}

NormFn norm_bwd_staged_ptr_f32(int vb, bool layer, int rows, bool full) {
    switch (vb) {
        case 16: return staged<16>(layer, rows, full);
        case 8: return staged<8>(layer, rows, full);
        case 4: return staged<4>(layer, rows, full);
        default: return nullptr;
    }
}

}  // namespace rmsnorm
