// rope.cu -- instances of the rotary kernels for any head_dim, strides and alignment.
#include "k_rope.cuh"

namespace rmsnorm {

template <typename T>
static RopeFn pick(bool interleaved, bool back) {
    if (interleaved) return back ? rope_any_kernel<T, true, true> : rope_any_kernel<T, true, false>;
    return back ? rope_any_kernel<T, false, true> : rope_any_kernel<T, false, false>;
}

RopeFn rope_any_ptr(int dtype, bool interleaved, bool back) {
    return dtype == 0 ? pick<float>(interleaved, back) : pick<__nv_bfloat16>(interleaved, back);
}
RopeFn rope_reduce_ptr() { return rope_reduce_kernel; }

}  // namespace rmsnorm
