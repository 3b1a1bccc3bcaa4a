// blocknorm.cu -- instances of the block boundary's kernels for any width.
#include "k_blocknorm.cuh"

namespace rmsnorm {

enum : int { kFwd, kRows, kCols };

template <typename T, int VB>
static BlockFn pick(int which) {
    switch (which) {
        case kFwd: return blocknorm_fwd_any_kernel<T, VB>;
        case kRows: return blocknorm_bwd_rows_kernel<T, VB>;
        default: return blocknorm_bwd_cols_kernel<T, VB>;
    }
}

template <typename T>
static BlockFn pick_vb(int vb, int which) {
    switch (vb) {
        case 16: return pick<T, 16>(which);
        case 8: return pick<T, 8>(which);
        case 4: return pick<T, 4>(which);
        default:
            if constexpr (sizeof(T) == 2) return pick<T, 2>(which);
            return nullptr;
    }
}

static BlockFn pick_all(int dtype, int vb, int which) {
    return dtype == 0 ? pick_vb<float>(vb, which) : pick_vb<__nv_bfloat16>(vb, which);
}

template <typename T>
static BlockFn pick_reduce(int width, bool gates) {
    if (width == 4) return gates ? blocknorm_reduce_kernel<T, 4, true> : blocknorm_reduce_kernel<T, 4, false>;
    return gates ? blocknorm_reduce_kernel<T, 1, true> : blocknorm_reduce_kernel<T, 1, false>;
}

BlockFn blocknorm_fwd_any_ptr(int dtype, int vb) { return pick_all(dtype, vb, kFwd); }
template <typename T, int VB>
static BlockFn pick_regs(int nv) {
    return nv == kBlockRegsVecs ? blocknorm_fwd_regs_kernel<T, VB, kBlockRegsVecs, true>
                                : blocknorm_fwd_regs_kernel<T, VB, 2 * kBlockRegsVecs, false>;
}
BlockFn blocknorm_fwd_regs_ptr(int dtype, int vb, int nv) {
    if (dtype == 0) return vb == 8 ? pick_regs<float, 8>(nv) : pick_regs<float, 4>(nv);
    return vb == 8 ? pick_regs<__nv_bfloat16, 8>(nv)
           : vb == 4 ? pick_regs<__nv_bfloat16, 4>(nv) : pick_regs<__nv_bfloat16, 2>(nv);
}
BlockFn blocknorm_bwd_rows_ptr(int dtype, int vb) { return pick_all(dtype, vb, kRows); }
BlockFn blocknorm_bwd_cols_ptr(int dtype, int vb) { return pick_all(dtype, vb, kCols); }
BlockFn blocknorm_reduce_ptr(int dtype, int width, bool gates) {
    return dtype == 0 ? pick_reduce<float>(width, gates) : pick_reduce<__nv_bfloat16>(width, gates);
}
int blocknorm_rows_block() { return kBlockRowsThreads; }
int blocknorm_cols_block() { return kBlockColsThreads; }

}  // namespace rmsnorm
