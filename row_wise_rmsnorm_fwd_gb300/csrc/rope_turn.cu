// rope_turn.cu -- instances of the vector kernel, kRopeTurn.
#include "rope_vec_pick.cuh"

namespace rmsnorm {

RopeFn rope_vec_ptr_turn(int dtype, int vb, bool interleaved) {
    return rope_pick_vec_all<kRopeTurn>(dtype, vb, interleaved);
}

}  // namespace rmsnorm
