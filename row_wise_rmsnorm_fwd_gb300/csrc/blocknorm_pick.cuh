// blocknorm_pick.cuh -- instances of the block boundary's staged kernels for one type.
#pragma once
#include "k_blocknorm_staged.cuh"

namespace rmsnorm {

template <typename T, bool BACK, bool POST, bool PRE, bool CL, int MODE, int VB = 16>
static BlockFn blocknorm_kernel() {
    if constexpr (BACK) return blocknorm_bwd_staged_kernel<T, POST, PRE, CL, MODE, VB>;
    else return blocknorm_fwd_staged_kernel<T, POST, PRE, CL, MODE, VB>;
}

template <typename T, bool BACK, bool POST, bool PRE>
static BlockFn blocknorm_pick(const BlockVariant& v) {
    if constexpr (POST || PRE) {
        if (v.whole && v.gate)
            return v.cluster ? blocknorm_kernel<T, BACK, POST, PRE, true, kBlockGated>()
                             : blocknorm_kernel<T, BACK, POST, PRE, false, kBlockGated>();
        if (v.whole)
            return v.cluster ? blocknorm_kernel<T, BACK, POST, PRE, true, kBlockPlain>()
                             : blocknorm_kernel<T, BACK, POST, PRE, false, kBlockPlain>();
    }
    return v.cluster ? blocknorm_kernel<T, BACK, POST, PRE, true, kBlockSome>()
                     : blocknorm_kernel<T, BACK, POST, PRE, false, kBlockSome>();
}

template <typename T, bool BACK>
static BlockFn blocknorm_pick_all(const BlockVariant& v) {
    if (v.post) return v.pre ? blocknorm_pick<T, BACK, true, true>(v) : blocknorm_pick<T, BACK, true, false>(v);
    return v.pre ? blocknorm_pick<T, BACK, false, true>(v) : blocknorm_pick<T, BACK, false, false>(v);
}

// Ragged rows.
template <typename T, bool BACK, int VB>
static BlockFn blocknorm_pick_ragged(const BlockVariant& v) {
    if (v.post) return v.pre ? blocknorm_kernel<T, BACK, true, true, false, kBlockSome, VB>()
                             : blocknorm_kernel<T, BACK, true, false, false, kBlockSome, VB>();
    return v.pre ? blocknorm_kernel<T, BACK, false, true, false, kBlockSome, VB>()
                 : blocknorm_kernel<T, BACK, false, false, false, kBlockSome, VB>();
}

template <typename T, bool BACK>
static BlockFn blocknorm_pick_ragged_all(const BlockVariant& v) {
    if (v.vb == 8) return blocknorm_pick_ragged<T, BACK, 8>(v);
    if (v.vb == 4) return blocknorm_pick_ragged<T, BACK, 4>(v);
    if constexpr (sizeof(T) == 2) return blocknorm_pick_ragged<T, BACK, 2>(v);
    return nullptr;
}

}  // namespace rmsnorm
