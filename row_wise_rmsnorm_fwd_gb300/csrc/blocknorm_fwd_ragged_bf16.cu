// blocknorm_fwd_ragged_bf16.cu -- instances of the block boundary's staged kernel for ragged rows,
// forward, bf16.
#include "blocknorm_pick.cuh"

namespace rmsnorm {

BlockFn blocknorm_fwd_ragged_bf16(const BlockVariant& v) { return blocknorm_pick_ragged_all<__nv_bfloat16, false>(v); }

}  // namespace rmsnorm
