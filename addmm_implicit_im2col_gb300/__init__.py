"""fp32 addmm and groups==1 NCHW conv2d as one tiled GEMM on sm_103a, 4-bit
(MXFP4) products, routing to experts, its balance loss and the experts' products,
low-rank adapters beside a projection.

The compute runs in the CUDA library ``libimc.so`` built from ``csrc/``;
``binding`` wraps its C ABI.  Importing this package does not load the
library: the first call into ``binding`` does, and raises if it is missing.
"""
__all__ = ["binding", "synth"]


def __getattr__(name):
    if name in ("addmm", "conv2d", "linear", "gemm_addmm_f32", "conv2d_gemm_f32", "linear_f32",
                "quantize_mxfp4", "dequantize_mxfp4", "linear_mxfp4", "linear_mxfp4_backward",
                "route_experts", "route_experts_backward", "experts_layout",
                "experts_linear_mxfp4", "experts_linear_mxfp4_backward", "experts_combine", "experts_combine_backward",
                "balance_loss", "balance_loss_backward", "adapters_linear", "adapters_linear_backward"):
        from . import binding
        return getattr(binding, name)
    raise AttributeError(name)
