// rope_back.cu -- instances of the vector kernel, kRopeTurnBack.
#include "rope_vec_pick.cuh"

namespace rmsnorm {

RopeFn rope_vec_ptr_back(int dtype, int vb, bool interleaved) {
    return rope_pick_vec_all<kRopeTurnBack>(dtype, vb, interleaved);
}

}  // namespace rmsnorm
