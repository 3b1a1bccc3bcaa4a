// blocknorm_fwd_bf16.cu -- instances of the block boundary's staged kernel, forward, bf16.
#include "blocknorm_pick.cuh"

namespace rmsnorm {

BlockFn blocknorm_fwd_staged_bf16(const BlockVariant& v) { return blocknorm_pick_all<__nv_bfloat16, false>(v); }

}  // namespace rmsnorm
