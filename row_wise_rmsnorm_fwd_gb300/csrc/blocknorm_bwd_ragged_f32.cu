// blocknorm_bwd_ragged_f32.cu -- instances of the block boundary's staged kernel for ragged rows,
// backward, fp32.
#include "blocknorm_pick.cuh"

namespace rmsnorm {

BlockFn blocknorm_bwd_ragged_f32(const BlockVariant& v) { return blocknorm_pick_ragged_all<float, true>(v); }

}  // namespace rmsnorm
