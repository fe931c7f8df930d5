"""B200-native dense GEMM: C = A.B with bf16 inputs / fp32 accumulation, and a
block-scaled MXFP8 variant, as hand-written sm_100a kernels behind a C ABI.

The binding (``gemm_bf16``, ``gemm_mxfp8``, ``gemm_check_device_status``,
``gemm_status_string`` ...) is loaded on first attribute access, so that
``synth`` can be imported on machines without the built library.  Accessing
a binding name when the library is missing raises immediately: there is no
fallback path.  A loaded name stays, so that later accesses cost nothing.
"""
from importlib import import_module

_BINDING_NAMES = {
    "gemm_bf16", "gemm_bf16_ex", "gemm_bf16_fused", "gemm_bf16_noalloc", "gemm_mxfp8", "gemm_rmsnorm",
    "gemm_rmsnorm_backward", "gemm_rmsnorm_backward_workspace", "gemm_mxfp8_quantize", "gemm_bf16_w4", "gemm_bf16_grouped",
    "gemm_bf16_grouped_wgrad", "gemm_fp4", "gemm_fp4_quantize", "gemm_fp4_scale_bytes", "FP4_MX", "FP4_NV",
    "gemm_check_device_status", "gemm_status_string",
    "gemm_force_config", "gemm_select_config", "gemm_launches_per_call",
    "gemm_last_timeout_detail", "GemmError", "OUT_F32", "OUT_BF16", "KMAJOR", "MNMAJOR", "ACT_NONE", "ACT_RELU",
    "ACT_GELU", "ACT_GELU_TANH", "CONFIGS",
    "STATUS_NAMES", "lib", "library_path",
}


def __getattr__(name):
    if name in _BINDING_NAMES:
        value = globals()[name] = getattr(import_module(".gemm", __name__), name)
        return value
    raise AttributeError(name)
