// blocknorm_fwd.cu -- instances of the block boundary's staged kernel, forward.
#include "k_blocknorm_staged.cuh"

namespace rmsnorm {

template <typename T, bool CL>
static BlockFn pick(bool post, bool pre) {
    if (post) return pre ? blocknorm_fwd_staged_kernel<T, true, true, CL> : blocknorm_fwd_staged_kernel<T, true, false, CL>;
    return pre ? blocknorm_fwd_staged_kernel<T, false, true, CL> : blocknorm_fwd_staged_kernel<T, false, false, CL>;
}

BlockFn blocknorm_fwd_staged_ptr(int dtype, bool post, bool pre, bool cluster) {
    if (dtype == 0) return cluster ? pick<float, true>(post, pre) : pick<float, false>(post, pre);
    return cluster ? pick<__nv_bfloat16, true>(post, pre) : pick<__nv_bfloat16, false>(post, pre);
}

}  // namespace rmsnorm
