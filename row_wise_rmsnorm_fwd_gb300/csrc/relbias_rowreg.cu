// relbias_rowreg.cu -- instances of the register-resident kernels of the row
// softmax with a relative position bias, both dtypes.
#include "k_relbias.cuh"

namespace rmsnorm {

template <typename T, int NV>
static BiasFn rowreg(bool shift, bool bwd) {
    if (bwd) return shift ? relbias_bwd_rowreg_kernel<T, NV, true> : relbias_bwd_rowreg_kernel<T, NV, false>;
    return shift ? relbias_fwd_rowreg_kernel<T, NV, true> : relbias_fwd_rowreg_kernel<T, NV, false>;
}

BiasFn relbias_rowreg_ptr(int dtype, int nv, bool shift, bool bwd) {
    if (nv == 4) return dtype == 0 ? rowreg<float, 4>(shift, bwd) : rowreg<__nv_bfloat16, 4>(shift, bwd);
    if (nv == 6) return dtype == 0 ? rowreg<float, 6>(shift, bwd) : rowreg<__nv_bfloat16, 6>(shift, bwd);
    return nullptr;
}

}  // namespace rmsnorm
