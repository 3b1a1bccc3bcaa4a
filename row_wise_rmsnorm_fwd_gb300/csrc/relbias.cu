// relbias.cu -- instances of the kernels of the row softmax with a relative
// position bias for rows of any width, both dtypes.
#include "k_relbias.cuh"

namespace rmsnorm {

template <typename T>
static BiasFn wide(int vb, bool bwd) {
    switch (vb) {
        case 16: return bwd ? relbias_bwd_wide_kernel<T, 16> : relbias_fwd_wide_kernel<T, 16>;
        case 8: return bwd ? relbias_bwd_wide_kernel<T, 8> : relbias_fwd_wide_kernel<T, 8>;
        case 4: return bwd ? relbias_bwd_wide_kernel<T, 4> : relbias_fwd_wide_kernel<T, 4>;
        case 2:
            if constexpr (sizeof(T) == 2)
                return bwd ? relbias_bwd_wide_kernel<T, 2> : relbias_fwd_wide_kernel<T, 2>;
            return nullptr;
        default: return nullptr;
    }
}

BiasFn relbias_fwd_wide_ptr(int dtype, int vb) {
    return dtype == 0 ? wide<float>(vb, false) : wide<__nv_bfloat16>(vb, false);
}
BiasFn relbias_bwd_wide_ptr(int dtype, int vb) {
    return dtype == 0 ? wide<float>(vb, true) : wide<__nv_bfloat16>(vb, true);
}
int relbias_wide_block() { return kBiasWideThreads; }
BiasFn relbias_reduce_ptr() { return relbias_reduce_kernel; }
int relbias_reduce_block() { return kBiasReduceThreads; }

}  // namespace rmsnorm
