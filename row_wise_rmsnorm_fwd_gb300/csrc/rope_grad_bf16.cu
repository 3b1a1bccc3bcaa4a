// rope_grad_bf16.cu -- instances of the rotary vector kernel, kRopeGrad, bf16.
#include "rope_vec_pick.cuh"

namespace rmsnorm {

RopeFn rope_vec_bf16_grad(int vb, bool interleaved, int lanes) {
    return rope_pick_vec_all<__nv_bfloat16, kRopeGrad>(vb, interleaved, lanes);
}

}  // namespace rmsnorm
