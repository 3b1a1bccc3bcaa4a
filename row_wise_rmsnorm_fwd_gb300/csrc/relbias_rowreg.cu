// relbias_rowreg.cu -- instances of the register-resident kernels of the row
// softmax with a relative position bias, both dtypes.
#include "k_relbias.cuh"

namespace rmsnorm {

static_assert(kBiasVecs * 16 == kBiasRowBytesPerThread, "a thread's bytes of a row");

BiasFn relbias_fwd_rowreg_ptr(int dtype, bool shift) {
    if (dtype == 0)
        return shift ? relbias_fwd_rowreg_kernel<float, true> : relbias_fwd_rowreg_kernel<float, false>;
    return shift ? relbias_fwd_rowreg_kernel<__nv_bfloat16, true>
                 : relbias_fwd_rowreg_kernel<__nv_bfloat16, false>;
}

BiasFn relbias_bwd_rowreg_ptr(int dtype, bool shift) {
    if (dtype == 0)
        return shift ? relbias_bwd_rowreg_kernel<float, true> : relbias_bwd_rowreg_kernel<float, false>;
    return shift ? relbias_bwd_rowreg_kernel<__nv_bfloat16, true>
                 : relbias_bwd_rowreg_kernel<__nv_bfloat16, false>;
}

}  // namespace rmsnorm
