// blocknorm_bwd_f32.cu -- instances of the block boundary's staged kernel, backward, fp32.
#include "blocknorm_pick.cuh"

namespace rmsnorm {

BlockFn blocknorm_bwd_staged_f32(const BlockVariant& v) { return blocknorm_pick_all<float, true>(v); }

}  // namespace rmsnorm
