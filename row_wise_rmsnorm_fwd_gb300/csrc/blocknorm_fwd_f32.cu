// blocknorm_fwd_f32.cu -- instances of the block boundary's staged kernel, forward, fp32.
#include "blocknorm_pick.cuh"

namespace rmsnorm {

BlockFn blocknorm_fwd_staged_f32(const BlockVariant& v) { return blocknorm_pick_all<float, false>(v); }

}  // namespace rmsnorm
