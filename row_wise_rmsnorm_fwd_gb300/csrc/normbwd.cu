// normbwd.cu -- instances of the norm backward kernels for any width.
#include "k_normbwd.cuh"

namespace rmsnorm {

template <typename T, bool LAYER>
static NormFn pick(int vb, bool cols) {
    switch (vb) {
        case 16: return cols ? norm_bwd_cols_kernel<T, 16, LAYER> : norm_bwd_rows_kernel<T, 16, LAYER>;
        case 8: return cols ? norm_bwd_cols_kernel<T, 8, LAYER> : norm_bwd_rows_kernel<T, 8, LAYER>;
        case 4: return cols ? norm_bwd_cols_kernel<T, 4, LAYER> : norm_bwd_rows_kernel<T, 4, LAYER>;
        case 2:
            if constexpr (sizeof(T) == 2)
                return cols ? norm_bwd_cols_kernel<T, 2, LAYER> : norm_bwd_rows_kernel<T, 2, LAYER>;
            return nullptr;
        default: return nullptr;
    }
}

static NormFn pick_all(int dtype, int vb, bool layer, bool cols) {
    if (dtype == 0) return layer ? pick<float, true>(vb, cols) : pick<float, false>(vb, cols);
    return layer ? pick<__nv_bfloat16, true>(vb, cols) : pick<__nv_bfloat16, false>(vb, cols);
}

NormFn norm_bwd_rows_ptr(int dtype, int vb, bool layer) { return pick_all(dtype, vb, layer, false); }
NormFn norm_bwd_cols_ptr(int dtype, int vb, bool layer) { return pick_all(dtype, vb, layer, true); }
NormFn norm_bwd_reduce_ptr(int width) {
    return width == 4 ? norm_bwd_reduce_kernel<4> : norm_bwd_reduce_kernel<1>;
}
int norm_bwd_rows_block() { return kBwdRowsThreads; }
int norm_bwd_cols_block() { return kBwdColsThreads; }

}  // namespace rmsnorm
