// blocknorm_fwd_ragged_f32.cu -- instances of the block boundary's staged kernel for ragged rows,
// forward, fp32.
#include "blocknorm_pick.cuh"

namespace rmsnorm {

BlockFn blocknorm_fwd_ragged_f32(const BlockVariant& v) { return blocknorm_pick_ragged_all<float, false>(v); }

}  // namespace rmsnorm
