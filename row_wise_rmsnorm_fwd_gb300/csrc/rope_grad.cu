// rope_grad.cu -- instances of the vector kernel, kRopeGrad.
#include "rope_vec_pick.cuh"

namespace rmsnorm {

RopeFn rope_vec_ptr_grad(int dtype, int vb, bool interleaved) {
    return rope_pick_vec_all<kRopeGrad>(dtype, vb, interleaved);
}

}  // namespace rmsnorm
