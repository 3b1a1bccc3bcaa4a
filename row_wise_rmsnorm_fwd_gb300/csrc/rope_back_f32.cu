// rope_back_f32.cu -- instances of the rotary vector kernel, kRopeTurnBack, fp32.
#include "rope_vec_pick.cuh"

namespace rmsnorm {

RopeFn rope_vec_f32_back(int vb, bool interleaved, int lanes) {
    return rope_pick_vec_all<float, kRopeTurnBack>(vb, interleaved, lanes);
}

}  // namespace rmsnorm
