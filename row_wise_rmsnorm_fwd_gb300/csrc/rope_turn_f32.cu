// rope_turn_f32.cu -- instances of the rotary vector kernel, kRopeTurn, fp32.
#include "rope_vec_pick.cuh"

namespace rmsnorm {

RopeFn rope_vec_f32_turn(int vb, bool interleaved, int lanes) {
    return rope_pick_vec_all<float, kRopeTurn>(vb, interleaved, lanes);
}

}  // namespace rmsnorm
