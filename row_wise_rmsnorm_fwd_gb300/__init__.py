"""librmsnorm: row-wise RMSNorm, layer norm and row softmax kernels for NVIDIA GB300.

``y[r, j] = (x[r, j] * rsqrt(mean_j x[r, j]^2 + eps)) * w[j]`` computed by
hand-written CUDA kernels behind a C ABI (``include/rmsnorm.h``).  This package
holds the CUDA sources (``csrc/``), their in-tree build (``build.py``), the
ctypes binding (``binding.py``) and the seeded workload generators
(``workloads.py``).  The binding is imported lazily so that the generators
can be used without the compiled library.
"""

_BINDING_NAMES = {
    "rmsnorm_fwd_f32", "rmsnorm_fwd_bf16", "rmsnorm_fwd_ex", "rmsnorm_plan",
    "rmsnorm_last_device_status", "rmsnorm_status_string", "rmsnorm_abi_version",
    "rmsnorm_last_cuda_error", "rowsoftmax_fwd_f32", "rowsoftmax_fwd_bf16",
    "rowsoftmax_fwd_ex", "rowsoftmax_plan",
    "rmsnorm_bwd_f32", "rmsnorm_bwd_bf16", "rmsnorm_bwd_ex", "rmsnorm_bwd_workspace",
    "layernorm_fwd_f32", "layernorm_fwd_bf16", "layernorm_fwd_ex",
    "layernorm_bwd_f32", "layernorm_bwd_bf16", "layernorm_bwd_ex", "layernorm_bwd_workspace",
    "rowsoftmax_relbias_fwd_f32", "rowsoftmax_relbias_fwd_bf16", "rowsoftmax_relbias_fwd_ex",
    "rowsoftmax_relbias_bwd_f32", "rowsoftmax_relbias_bwd_bf16", "rowsoftmax_relbias_bwd_ex",
    "rowsoftmax_relbias_bwd_workspace", "rowsoftmax_relbias_bucket",
    "make_options", "RmsnormError", "raw", "load",
}


def __getattr__(name):
    if name in _BINDING_NAMES:
        from . import binding
        return getattr(binding, name)
    raise AttributeError(name)
