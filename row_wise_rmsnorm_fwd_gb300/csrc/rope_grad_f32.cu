// rope_grad_f32.cu -- instances of the rotary vector kernel, kRopeGrad, fp32.
#include "rope_vec_pick.cuh"

namespace rmsnorm {

RopeFn rope_vec_f32_grad(int vb, bool interleaved, int lanes) {
    return rope_pick_vec_all<float, kRopeGrad>(vb, interleaved, lanes);
}

}  // namespace rmsnorm
