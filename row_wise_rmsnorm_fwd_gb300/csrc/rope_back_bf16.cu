// rope_back_bf16.cu -- instances of the rotary vector kernel, kRopeTurnBack, bf16.
#include "rope_vec_pick.cuh"

namespace rmsnorm {

RopeFn rope_vec_bf16_back(int vb, bool interleaved, int lanes) {
    return rope_pick_vec_all<__nv_bfloat16, kRopeTurnBack>(vb, interleaved, lanes);
}

}  // namespace rmsnorm
