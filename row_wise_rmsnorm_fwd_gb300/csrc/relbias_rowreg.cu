// relbias_rowreg.cu -- instances of the register-resident kernels of the row
// softmax with a relative position bias, both dtypes.
#include "k_relbias.cuh"

namespace rmsnorm {

template <typename T, int NV, bool SHIFT>
static BiasFn rowreg(bool bwd, bool turns) {
    if (!bwd) return relbias_fwd_rowreg_kernel<T, NV, SHIFT>;
    return turns ? relbias_bwd_rowreg_kernel<T, NV, SHIFT, true> : relbias_bwd_rowreg_kernel<T, NV, SHIFT, false>;
}

template <typename T>
static BiasFn rowreg(int nv, bool shift, bool bwd, bool turns) {
    if (nv == 4) return shift ? rowreg<T, 4, true>(bwd, turns) : rowreg<T, 4, false>(bwd, turns);
    if (nv == 6) return shift ? rowreg<T, 6, true>(bwd, turns) : rowreg<T, 6, false>(bwd, turns);
    return nullptr;
}

BiasFn relbias_rowreg_ptr(int dtype, int nv, bool shift, bool bwd, bool turns) {
    return dtype == 0 ? rowreg<float>(nv, shift, bwd, turns) : rowreg<__nv_bfloat16>(nv, shift, bwd, turns);
}

}  // namespace rmsnorm
