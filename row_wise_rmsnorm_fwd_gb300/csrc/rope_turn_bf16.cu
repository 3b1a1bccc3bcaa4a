// rope_turn_bf16.cu -- instances of the rotary vector kernel, kRopeTurn, bf16.
#include "rope_vec_pick.cuh"

namespace rmsnorm {

RopeFn rope_vec_bf16_turn(int vb, bool interleaved, int lanes) {
    return rope_pick_vec_all<__nv_bfloat16, kRopeTurn>(vb, interleaved, lanes);
}

}  // namespace rmsnorm
