"""Python binding of libimc's C ABI (include/imc.h).

The functions named like the C entry points take raw integer device pointers
and return the C status code.  ``addmm`` and ``conv2d`` wrap them for torch
CUDA tensors (PyTorch supplies device memory and the current stream only;
every step of the computation runs in libimc's kernels).  There is no CPU
fallback: the library must be built (``python -m addmm_implicit_im2col_gb300.build``)
and loading it raises otherwise.
"""
from __future__ import annotations

import ctypes
import functools
import importlib
import os
import sys
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libimc.so")

IMC_OK = 0
IMC_ERR_NULL = -1
IMC_ERR_SHAPE = -2
IMC_ERR_ARG = -3
IMC_ERR_ALIAS = -4
IMC_ERR_CUDA = -5
IMC_ERR_TIMEOUT = -6
IMC_ERR_DEVICE = -7
IMC_ERR_SCRATCH = -8
NOALLOC_SCRATCH_BYTES = 32 << 20

MODES = {"default": 0, "tf32": 1, "simt": 2, "force_tc3": 3, "force_tc1": 4, "direct": 5}
ACT_RELU = 0x100
KERNELS = {0: "none", 1: "tc3", 2: "tc1", 3: "simt", 4: "fill", 5: "direct", 6: "mxfp4",
           7: "experts", 8: "adapters"}
F32, F16, BF16, MXFP4 = 0, 1, 2, 3
SCORES = {"softmax": 0, "sigmoid": 1}

# Every symbol the header declares, with (restype, argtypes).
_i64, _dbl, _vp, _int = ctypes.c_int64, ctypes.c_double, ctypes.c_void_p, ctypes.c_int
SIGNATURES = {
    "gemm_addmm_f32": (_int, [_vp, _int, _vp, _vp, _vp, _i64, _i64, _i64, _dbl, _dbl, _vp]),
    "gemm_addmm_f32_ex": (_int, [_vp, _int, _vp, _vp, _vp, _i64, _i64, _i64, _dbl, _dbl, _int,
                                 _vp]),
    "conv2d_gemm_f32": (_int, [_vp, _vp, _vp, _vp] + [_i64] * 10 + [_vp]),
    "conv2d_gemm_f32_ex": (_int, [_vp, _vp, _vp, _vp] + [_i64] * 10 + [_int, _vp]),
    "conv2d_gemm_f32_nd": (_int, [_vp, _vp, _vp, _vp] + [_i64] * 13 + [_int, _vp]),
    "gemm_addmm_f32_ws": (_int, [_vp, _int, _vp, _vp, _vp, _i64, _i64, _i64, _dbl, _dbl, _int,
                                 _vp, ctypes.c_size_t, _vp]),
    "gemm_addmm_f32_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64, _int]),
    "conv2d_gemm_f32_ws": (_int, [_vp, _vp, _vp, _vp] + [_i64] * 13 + [_int, _vp, ctypes.c_size_t,
                                                                      _vp]),
    "conv2d_gemm_f32_workspace_bytes": (ctypes.c_size_t, [_i64] * 13 + [_int]),
    "gemm_addmm_f32_noalloc": (_int, [_vp, _int, _vp, _vp, _vp, _i64, _i64, _i64, _dbl, _dbl,
                                      _int, _vp]),
    "linear_f32": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp]),
    "linear_f32_ws": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, ctypes.c_size_t, _vp]),
    "linear_f32_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64, _int]),
    "gemm_addmm_f32_host": (_int, [_vp, _int, _vp, _vp, _vp, _i64, _i64, _i64, _dbl, _dbl, _int,
                                   _vp]),
    "conv2d_gemm_f32_host": (_int, [_vp, _vp, _vp, _vp] + [_i64] * 13 + [_int, _vp]),
    "mxfp4_bytes": (ctypes.c_size_t, [_i64] * 3),
    "mxfp4_quantize": (_int, [_vp, _int] + [_i64] * 5 + [_int, _vp, _vp]),
    "mxfp4_dequantize": (_int, [_vp] + [_i64] * 3 + [_int, _vp, _vp]),
    "mxfp4_linear_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _int]),
    "mxfp4_linear": (_int, [_vp, _int, _i64, _vp, _vp, _vp, _int, _i64, _i64, _i64, _int, _vp,
                            ctypes.c_size_t, _vp]),
    "mxfp4_linear_backward_workspace_bytes": (ctypes.c_size_t, [_i64] * 3),
    "mxfp4_linear_backward": (_int, [_vp, _vp, _vp, _int, _i64, _i64, _i64, _vp, _vp, _vp,
                                     ctypes.c_size_t, _vp]),
    "moe_route": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _i64, _int, _i64, _i64, _int, _dbl, _vp,
                         _vp, _vp]),
    "moe_route_backward": (_int, [_vp, _vp, _int, _i64, _i64, _i64, _vp, _i64, _int, _int, _dbl,
                                  _vp, _vp]),
    "moe_layout_size": (_i64, [_i64] * 3),
    "moe_layout": (_int, [_vp, _i64, _i64, _i64, _vp, _vp]),
    "mxfp4_experts_linear_workspace_bytes": (ctypes.c_size_t, [_i64] * 4),
    "mxfp4_experts_linear": (_int, [_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp, _int] + [_i64] * 5
                             + [_int, _vp, ctypes.c_size_t, _vp]),
    "mxfp4_experts_weight_grad_workspace_bytes": (ctypes.c_size_t, [_i64] * 5),
    "mxfp4_experts_weight_grad": (_int, [_vp, _vp, _int, _i64, _vp, _vp] + [_i64] * 5
                                  + [_vp, ctypes.c_size_t, _vp]),
    "moe_combine": (_int, [_vp, _int, _vp, _i64, _i64, _i64, _vp, _vp]),
    "moe_combine_f32": (_int, [_vp, _vp, _i64, _i64, _i64, _vp, _int, _vp]),
    "moe_combine_backward": (_int, [_vp, _vp, _int, _vp, _i64, _i64, _i64, _vp, _vp, _vp]),
    "moe_balance_workspace_bytes": (ctypes.c_size_t, [_i64] * 3),
    "moe_balance": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _i64, _int, _vp, _i64, _vp, _vp, _vp,
                           ctypes.c_size_t, _vp]),
    "moe_balance_backward": (_int, [_vp, _vp, _int, _i64, _i64, _i64, _vp, _i64, _int, _vp, _vp,
                                    _i64, _vp, _int, _dbl, _vp, _vp]),
    "lowrank_linear_workspace_bytes": (ctypes.c_size_t, [_i64] * 3),
    "lowrank_linear": (_int, [_vp, _int, _i64] + [_vp] * 6 + [_i64] * 5
                       + [_vp, ctypes.c_size_t, _vp]),
    "lowrank_linear_backward_workspace_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "lowrank_linear_backward": (_int, [_vp] * 4 + [_int] + [_vp] * 6 + [_i64] * 5
                                 + [_vp, ctypes.c_size_t, _vp]),
    "imc_status_string": (ctypes.c_char_p, [_int]),
    "imc_last_kernel": (_int, []),
    "imc_last_kernel_name": (ctypes.c_char_p, []),
    "imc_launch_count": (ctypes.c_uint64, []),
    "imc_check_device_error": (_int, [_vp]),
    "imc_version": (_int, []),
    "imc_release_memory": (_int, []),
    "imc_selftest_wait_timeout": (_int, [_int, _vp]),
}

_lock = threading.Lock()
_lib = None


class ImcError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})" if what else
                         f"{status_string(status)} ({status})")


def load(path: str | None = None):
    """Loads libimc.so (once) and declares every exported signature."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise ImportError(f"{p} is not built; run python -m addmm_implicit_im2col_gb300.build")
        lib = ctypes.CDLL(p)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _lib = lib
        return lib


# ------------------------------------------------------ raw C-ABI mirrors
def gemm_addmm_f32(self, self_2d, mat1, mat2, out, M, N, K, beta, alpha, stream) -> int:
    return load().gemm_addmm_f32(self, self_2d, mat1, mat2, out, M, N, K, beta, alpha, stream)


def gemm_addmm_f32_ex(self, self_2d, mat1, mat2, out, M, N, K, beta, alpha, mode, stream) -> int:
    return load().gemm_addmm_f32_ex(self, self_2d, mat1, mat2, out, M, N, K, beta, alpha, mode,
                                    stream)


def gemm_addmm_f32_ws(self, self_2d, mat1, mat2, out, M, N, K, beta, alpha, mode, workspace,
                      workspace_bytes, stream) -> int:
    return load().gemm_addmm_f32_ws(self, self_2d, mat1, mat2, out, M, N, K, beta, alpha, mode,
                                    workspace, workspace_bytes, stream)


def gemm_addmm_f32_noalloc(self, self_2d, mat1, mat2, out, M, N, K, beta, alpha, mode,
                           stream) -> int:
    """The addmm entry point that allocates nothing (fixed library buffer)."""
    return load().gemm_addmm_f32_noalloc(self, self_2d, mat1, mat2, out, M, N, K, beta, alpha,
                                         mode, stream)


def gemm_addmm_f32_workspace_bytes(M, N, K, mode) -> int:
    return int(load().gemm_addmm_f32_workspace_bytes(M, N, K, mode))


def conv2d_gemm_f32(x, w, bias, out, B, IC, H, W, OC, KH, KW, stride, pad, dilation,
                    stream) -> int:
    return load().conv2d_gemm_f32(x, w, bias, out, B, IC, H, W, OC, KH, KW, stride, pad,
                                  dilation, stream)


def conv2d_gemm_f32_ex(x, w, bias, out, B, IC, H, W, OC, KH, KW, stride, pad, dilation, mode,
                       stream) -> int:
    return load().conv2d_gemm_f32_ex(x, w, bias, out, B, IC, H, W, OC, KH, KW, stride, pad,
                                     dilation, mode, stream)


def conv2d_gemm_f32_nd(x, w, bias, out, B, IC, H, W, OC, KH, KW, sH, sW, pH, pW, dH, dW, mode,
                       stream) -> int:
    return load().conv2d_gemm_f32_nd(x, w, bias, out, B, IC, H, W, OC, KH, KW, sH, sW, pH, pW,
                                     dH, dW, mode, stream)


def conv2d_gemm_f32_ws(x, w, bias, out, B, IC, H, W, OC, KH, KW, sH, sW, pH, pW, dH, dW, mode,
                       workspace, workspace_bytes, stream) -> int:
    return load().conv2d_gemm_f32_ws(x, w, bias, out, B, IC, H, W, OC, KH, KW, sH, sW, pH, pW,
                                     dH, dW, mode, workspace, workspace_bytes, stream)


def conv2d_gemm_f32_workspace_bytes(B, IC, H, W, OC, KH, KW, sH, sW, pH, pW, dH, dW,
                                    mode) -> int:
    return int(load().conv2d_gemm_f32_workspace_bytes(B, IC, H, W, OC, KH, KW, sH, sW, pH, pW,
                                                      dH, dW, mode))


def linear_f32(x, w, bias, out, M, N, K, mode, stream) -> int:
    return load().linear_f32(x, w, bias, out, M, N, K, mode, stream)


def linear_f32_ws(x, w, bias, out, M, N, K, mode, workspace, workspace_bytes, stream) -> int:
    return load().linear_f32_ws(x, w, bias, out, M, N, K, mode, workspace, workspace_bytes, stream)


def linear_f32_workspace_bytes(M, N, K, mode) -> int:
    return int(load().linear_f32_workspace_bytes(M, N, K, mode))


def gemm_addmm_f32_host(self, self_2d, mat1, mat2, out, M, N, K, beta, alpha, mode,
                        stream) -> int:
    return load().gemm_addmm_f32_host(self, self_2d, mat1, mat2, out, M, N, K, beta, alpha, mode,
                                      stream)


def conv2d_gemm_f32_host(x, w, bias, out, B, IC, H, W, OC, KH, KW, sH, sW, pH, pW, dH, dW, mode,
                         stream) -> int:
    return load().conv2d_gemm_f32_host(x, w, bias, out, B, IC, H, W, OC, KH, KW, sH, sW, pH, pW,
                                       dH, dW, mode, stream)


def mxfp4_bytes(batch, rows, cols) -> int:
    return int(load().mxfp4_bytes(batch, rows, cols))


def mxfp4_quantize(x, dtype, batch, rows, cols, batch_stride, row_stride, transpose, q,
                   stream) -> int:
    return load().mxfp4_quantize(x, dtype, batch, rows, cols, batch_stride, row_stride, transpose,
                                 q, stream)


def mxfp4_dequantize(q, batch, rows, cols, dtype, out, stream) -> int:
    return load().mxfp4_dequantize(q, batch, rows, cols, dtype, out, stream)


def mxfp4_linear_workspace_bytes(M, K, x_dtype) -> int:
    return int(load().mxfp4_linear_workspace_bytes(M, K, x_dtype))


def mxfp4_linear(x, x_dtype, row_stride, w, bias, out, out_dtype, M, N, K, flags, workspace,
                 workspace_bytes, stream) -> int:
    return load().mxfp4_linear(x, x_dtype, row_stride, w, bias, out, out_dtype, M, N, K, flags,
                               workspace, workspace_bytes, stream)


def mxfp4_linear_backward_workspace_bytes(M, N, K) -> int:
    return int(load().mxfp4_linear_backward_workspace_bytes(M, N, K))


def mxfp4_linear_backward(grad, x, w, dtype, M, N, K, grad_x, grad_w, workspace, workspace_bytes,
                          stream) -> int:
    return load().mxfp4_linear_backward(grad, x, w, dtype, M, N, K, grad_x, grad_w, workspace,
                                        workspace_bytes, stream)


def moe_route(logits, dtype, T, E, row_stride, bias, k, score, groups, top_groups, renormalize,
              scale, weights, experts, stream) -> int:
    return load().moe_route(logits, dtype, T, E, row_stride, bias, k, score, groups, top_groups,
                            renormalize, scale, weights, experts, stream)


def moe_route_backward(grad_weights, logits, dtype, T, E, row_stride, experts, k, score,
                       renormalize, scale, grad_logits, stream) -> int:
    return load().moe_route_backward(grad_weights, logits, dtype, T, E, row_stride, experts, k,
                                     score, renormalize, scale, grad_logits, stream)


def moe_layout_size(T, k, E) -> int:
    return int(load().moe_layout_size(T, k, E))


def moe_layout(experts, T, k, E, layout, stream) -> int:
    return load().moe_layout(experts, T, k, E, layout, stream)


def mxfp4_experts_linear_workspace_bytes(T, k, E, K) -> int:
    return int(load().mxfp4_experts_linear_workspace_bytes(T, k, E, K))


def mxfp4_experts_linear(x, x_dtype, x_rows, row_stride, w, bias, layout, out, out_dtype, T, k, E,
                         N, K, flags, workspace, workspace_bytes, stream) -> int:
    return load().mxfp4_experts_linear(x, x_dtype, x_rows, row_stride, w, bias, layout, out,
                                       out_dtype, T, k, E, N, K, flags, workspace,
                                       workspace_bytes, stream)


def mxfp4_experts_weight_grad_workspace_bytes(T, k, E, N, K) -> int:
    return int(load().mxfp4_experts_weight_grad_workspace_bytes(T, k, E, N, K))


def mxfp4_experts_weight_grad(grad, x, dtype, x_rows, layout, grad_w, T, k, E, N, K, workspace,
                              workspace_bytes, stream) -> int:
    return load().mxfp4_experts_weight_grad(grad, x, dtype, x_rows, layout, grad_w, T, k, E, N, K,
                                            workspace, workspace_bytes, stream)


def moe_combine(y, dtype, weights, T, k, N, out, stream) -> int:
    return load().moe_combine(y, dtype, weights, T, k, N, out, stream)


def moe_combine_f32(y, weights, T, k, N, out, out_dtype, stream) -> int:
    return load().moe_combine_f32(y, weights, T, k, N, out, out_dtype, stream)


def moe_combine_backward(grad, y, dtype, weights, T, k, N, grad_y, grad_weights, stream) -> int:
    return load().moe_combine_backward(grad, y, dtype, weights, T, k, N, grad_y, grad_weights,
                                       stream)


def moe_balance_workspace_bytes(T, S, E) -> int:
    return int(load().moe_balance_workspace_bytes(T, S, E))


def moe_balance(logits, dtype, T, E, row_stride, experts, k, score, offsets, S, loss, counts,
                workspace, workspace_bytes, stream) -> int:
    return load().moe_balance(logits, dtype, T, E, row_stride, experts, k, score, offsets, S, loss,
                              counts, workspace, workspace_bytes, stream)


def moe_balance_backward(grad_loss, logits, dtype, T, E, row_stride, experts, k, score, counts,
                         offsets, S, grad_weights, renormalize, scale, grad_logits, stream) -> int:
    return load().moe_balance_backward(grad_loss, logits, dtype, T, E, row_stride, experts, k,
                                       score, counts, offsets, S, grad_weights, renormalize, scale,
                                       grad_logits, stream)


def lowrank_linear_workspace_bytes(T, L, r) -> int:
    return int(load().lowrank_linear_workspace_bytes(T, L, r))


def lowrank_linear(x, dtype, row_stride, a, b, scale, layout, base, out, T, L, r, K, N, workspace,
                   workspace_bytes, stream) -> int:
    return load().lowrank_linear(x, dtype, row_stride, a, b, scale, layout, base, out, T, L, r, K,
                                 N, workspace, workspace_bytes, stream)


def lowrank_linear_backward_workspace_bytes(T, r) -> int:
    return int(load().lowrank_linear_backward_workspace_bytes(T, r))


def lowrank_linear_backward(grad, x, a, b, dtype, scale, layout, base, grad_x, grad_a, grad_b, T,
                            L, r, K, N, workspace, workspace_bytes, stream) -> int:
    return load().lowrank_linear_backward(grad, x, a, b, dtype, scale, layout, base, grad_x, grad_a,
                                          grad_b, T, L, r, K, N, workspace, workspace_bytes, stream)


def selftest_wait_timeout(limit_us, stream=None) -> int:
    return load().imc_selftest_wait_timeout(int(limit_us), stream)


def release_memory() -> int:
    return load().imc_release_memory()


def status_string(status: int) -> str:
    return load().imc_status_string(status).decode()


def last_kernel() -> str:
    return KERNELS.get(load().imc_last_kernel(), "unknown")


def last_kernel_name() -> str:
    """Name and form of the main kernel of this thread's last successful call."""
    return load().imc_last_kernel_name().decode()


def launch_count() -> int:
    return int(load().imc_launch_count())


def check_device_error(stream=None) -> int:
    return load().imc_check_device_error(stream)


# ------------------------------------------------------- torch-level API
def _stream_ptr(device):
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_tensor(t, name, ndim=None, host=False):
    import torch
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    where = "CPU" if host else "CUDA"
    placed = t.device.type == "cpu" if host else t.is_cuda
    if not placed or t.dtype != torch.float32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 {where} tensor")
    if ndim is not None and t.dim() not in ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def _mode(mode, relu):
    return MODES[mode] | (ACT_RELU if relu else 0)


def _addmm_dims(self, mat1, mat2, host):
    _check_tensor(mat1, "mat1", (2,), host)
    _check_tensor(mat2, "mat2", (2,), host)
    _check_tensor(self, "self", (1, 2), host)
    M, K = mat1.shape
    K2, N = mat2.shape
    if K2 != K:
        raise ValueError(f"mat2 must be [K, N] = [{K}, N], got {list(mat2.shape)}")
    self_2d = 0
    if self is not None:
        if self.dim() == 2:
            if list(self.shape) != [M, N]:
                raise ValueError("a 2-D self must be [M, N]")
            self_2d = 1
        elif self.shape[0] != N:
            raise ValueError("a 1-D self must be [N]")
    return M, N, K, self_2d


def _aligned16(t):
    return t.data_ptr() % 16 == 0


def addmm(self, mat1, mat2, *, beta=1.0, alpha=1.0, mode="default", relu=False, out=None):
    """out = beta*self + alpha*(mat1 @ mat2) on the GPU (aten.addmm semantics).

    self is [N] or [M, N]; alpha and beta default to 1.0.  ``mode`` is one of
    ``MODES``; ``relu`` fuses max(v, 0) into the epilogue.  Returns ``out``
    (allocated with torch when not given).
    """
    import torch
    M, N, K, self_2d = _addmm_dims(self, mat1, mat2, host=False)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=mat1.device)
    else:
        _check_tensor(out, "out", (2,))
    # scratch for the transposed mat2 comes from torch's allocator; the size
    # query assumes 16-byte aligned operands, and imc.h documents the extra
    # mat1 copy (M * Kp * 4 bytes) an unaligned mat1 needs
    nbytes = gemm_addmm_f32_workspace_bytes(M, N, K, MODES[mode])
    if nbytes and K % 4 == 0 and not _aligned16(mat1):
        nbytes += M * K * 4 + 256
    ws = torch.empty(nbytes, dtype=torch.uint8, device=mat1.device) if nbytes else None
    rc = gemm_addmm_f32_ws(_ptr(self), self_2d, _ptr(mat1), _ptr(mat2), _ptr(out), M, N, K,
                           float(beta), float(alpha), _mode(mode, relu), _ptr(ws), nbytes,
                           _stream_ptr(mat1.device))
    if rc != IMC_OK:
        raise ImcError(rc, "gemm_addmm_f32")
    return out


def linear(x, w, bias=None, *, mode="default", relu=False, out=None):
    """out = x @ w^T (+ bias) on the GPU (aten.linear semantics).

    x is [M, K], w is [N, K] (the transposed weight), bias [N] or None.
    """
    import torch
    _check_tensor(x, "x", (2,))
    _check_tensor(w, "w", (2,))
    _check_tensor(bias, "bias", (1,))
    M, K = x.shape
    N, K2 = w.shape
    if K2 != K:
        raise ValueError(f"w must be [N, K] = [N, {K}], got {list(w.shape)}")
    if bias is not None and bias.shape[0] != N:
        raise ValueError("bias must be [N]")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=x.device)
    else:
        _check_tensor(out, "out", (2,))
    nbytes = linear_f32_workspace_bytes(M, N, K, MODES[mode])
    if MODES[mode] != MODES["simt"] and K % 4 == 0:
        # the size query assumes 16-byte aligned operands; imc.h documents the
        # copies an unaligned x (M * Kp * 4) or weight (hi and lo, 2 * N * Kp * 4)
        # needs
        if not _aligned16(x):
            nbytes += M * K * 4 + 256
        if not _aligned16(w):
            nbytes += 2 * N * K * 4 + 256
    ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if nbytes else None
    rc = linear_f32_ws(_ptr(x), _ptr(w), _ptr(bias), _ptr(out), M, N, K, _mode(mode, relu),
                       _ptr(ws), nbytes, _stream_ptr(x.device))
    if rc != IMC_OK:
        raise ImcError(rc, "linear_f32")
    return out


def conv_out_size(n, k, stride, pad, dil) -> int:
    span = n + 2 * pad - dil * (k - 1) - 1
    return -1 if span < 0 else span // stride + 1


def _pair(v):
    return (int(v[0]), int(v[1])) if isinstance(v, (tuple, list)) else (int(v), int(v))


def _conv_dims(x, w, bias, stride, padding, dilation, host):
    _check_tensor(x, "x", (4,), host)
    _check_tensor(w, "w", (4,), host)
    _check_tensor(bias, "bias", (1,), host)
    B, IC, H, W = x.shape
    OC, IC2, KH, KW = w.shape
    if IC2 != IC:
        raise ValueError("weight must be [OC, IC, KH, KW] with the input's IC (groups == 1)")
    if bias is not None and bias.shape[0] != OC:
        raise ValueError("bias must be [OC]")
    sH, sW = _pair(stride)
    pH, pW = _pair(padding)
    dH, dW = _pair(dilation)
    OH = conv_out_size(H, KH, sH, pH, dH)
    OW = conv_out_size(W, KW, sW, pW, dW)
    if OH < 1 or OW < 1:
        raise ValueError("empty convolution output")
    return B, IC, H, W, OC, KH, KW, sH, sW, pH, pW, dH, dW, OH, OW


def conv2d(x, w, bias=None, stride=1, padding=0, dilation=1, *, mode="default", relu=False,
           out=None):
    """groups==1 NCHW conv2d via the implicit-im2col GEMM.

    x [B, IC, H, W], w [OC, IC, KH, KW], bias [OC] or None; stride, padding and
    dilation are ints or (h, w) pairs.  Returns out [B, OC, OH, OW].
    """
    import torch
    B, IC, H, W, OC, KH, KW, sH, sW, pH, pW, dH, dW, OH, OW = _conv_dims(
        x, w, bias, stride, padding, dilation, host=False)
    if out is None:
        out = torch.empty((B, OC, OH, OW), dtype=torch.float32, device=x.device)
    else:
        _check_tensor(out, "out", (4,))
    nbytes = conv2d_gemm_f32_workspace_bytes(B, IC, H, W, OC, KH, KW, sH, sW, pH, pW, dH, dW,
                                             MODES[mode])
    ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if nbytes else None
    rc = conv2d_gemm_f32_ws(_ptr(x), _ptr(w), _ptr(bias), _ptr(out), B, IC, H, W, OC, KH, KW,
                            sH, sW, pH, pW, dH, dW, _mode(mode, relu), _ptr(ws), nbytes,
                            _stream_ptr(x.device))
    if rc != IMC_OK:
        raise ImcError(rc, "conv2d_gemm_f32")
    return out


# ------------------------------------------------- host-buffer entry points
def _host_stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def addmm_host(self, mat1, mat2, *, beta=1.0, alpha=1.0, mode="default", relu=False, out=None,
               stream=None):
    """addmm on CPU tensors through gemm_addmm_f32_host: the library copies the
    inputs to the GPU, computes there and copies ``out`` back, all enqueued on
    ``stream`` (a torch.cuda.Stream; None: the current stream).  Returns ``out``
    at once; it holds the result after ``stream.synchronize()``.  Page-locked
    tensors (``pin_memory()``) let the copies run asynchronously.
    """
    import torch
    M, N, K, self_2d = _addmm_dims(self, mat1, mat2, host=True)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, pin_memory=mat1.is_pinned())
    else:
        _check_tensor(out, "out", (2,), host=True)
    rc = gemm_addmm_f32_host(_ptr(self), self_2d, _ptr(mat1), _ptr(mat2), _ptr(out), M, N, K,
                             float(beta), float(alpha), _mode(mode, relu), _host_stream(stream))
    if rc != IMC_OK:
        raise ImcError(rc, "gemm_addmm_f32_host")
    return out


def conv2d_host(x, w, bias=None, stride=1, padding=0, dilation=1, *, mode="default", relu=False,
                out=None, stream=None):
    """conv2d on CPU tensors through conv2d_gemm_f32_host (as ``addmm_host``)."""
    import torch
    B, IC, H, W, OC, KH, KW, sH, sW, pH, pW, dH, dW, OH, OW = _conv_dims(
        x, w, bias, stride, padding, dilation, host=True)
    if out is None:
        out = torch.empty((B, OC, OH, OW), dtype=torch.float32, pin_memory=x.is_pinned())
    else:
        _check_tensor(out, "out", (4,), host=True)
    rc = conv2d_gemm_f32_host(_ptr(x), _ptr(w), _ptr(bias), _ptr(out), B, IC, H, W, OC, KH, KW,
                              sH, sW, pH, pW, dH, dW, _mode(mode, relu), _host_stream(stream))
    if rc != IMC_OK:
        raise ImcError(rc, "conv2d_gemm_f32_host")
    return out


# ---------------------------- 4-bit products, experts and adapters (torch level)
# These calls take a few microseconds on the GPU when a model decodes, so their
# wrappers avoid what costs microseconds on the host: repeated imports, stream
# objects, a library call for a size that was asked for before.
#
# They record nothing for autograd (a result of a tensor that requires grad is
# detached, as with the fp32 calls): a training step calls the *_backward functions.
# All tensors of a call are on the current device.
_torch = None
_raw_stream = None
_current_device = None
_calls = None  # the C entry points without ctypes (csrc/calls.c), else this module's mirrors
_DTYPE_IDS = {}
_size = functools.lru_cache(maxsize=4096)(mxfp4_bytes)
_linear_size = functools.lru_cache(maxsize=4096)(mxfp4_linear_workspace_bytes)
_layout_size = functools.lru_cache(maxsize=4096)(moe_layout_size)
_experts_size = functools.lru_cache(maxsize=4096)(mxfp4_experts_linear_workspace_bytes)
_balance_size = functools.lru_cache(maxsize=4096)(moe_balance_workspace_bytes)
_lowrank_size = functools.lru_cache(maxsize=4096)(lowrank_linear_workspace_bytes)
_lowrank_back_size = functools.lru_cache(maxsize=4096)(lowrank_linear_backward_workspace_bytes)
_backward_size = functools.lru_cache(maxsize=4096)(mxfp4_linear_backward_workspace_bytes)


def _setup():
    """Imports torch and loads the library, once."""
    global _torch, _calls, _raw_stream, _current_device
    if _torch is None:
        import torch
        _DTYPE_IDS.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})
        load()
        try:
            calls = importlib.import_module(__package__ + "._calls")
        except ModuleNotFoundError:  # built without Python's headers
            calls = sys.modules[__name__]
        _raw_stream = torch._C._cuda_getCurrentRawStream
        _current_device = torch._C._cuda_getDevice
        _calls, _torch = calls, torch
    return _torch


def _dtype_id(dtype, name):
    try:
        return _DTYPE_IDS[dtype]
    except KeyError:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {dtype}") from None


def _rows_of(t, name, ndim=2):
    """Type id, shape and strides of a CUDA tensor of a float type with contiguous last dimension."""
    if not isinstance(t, (_torch or _setup()).Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if not t.is_cuda or len(shape) != ndim:
        raise ValueError(f"{name} must be a CUDA tensor of {ndim} dimensions")
    stride = t.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    dt = _DTYPE_IDS.get(t.dtype)
    if dt is None:
        _dtype_id(t.dtype, name)
    return dt, shape, (stride if shape[-2] > 1 else stride[:-2] + (shape[-1], 1))


def _check_plain(t, name, dtype, shape, like):
    """A contiguous CUDA tensor of this type and shape on the device of `like`."""
    if t is None:
        return
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if (not t.is_cuda or t.dtype != dtype or not t.is_contiguous()
            or (t is not like and t.device != like.device)):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on {like.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _check_buffer(data, dtype, count):
    """A one-dimensional contiguous tensor of this type with `count` values at least."""
    if not isinstance(data, _torch.Tensor):
        raise TypeError("data must be a torch.Tensor")
    if data.dtype != dtype or data.dim() != 1 or not data.is_contiguous() or data.numel() < count:
        raise ValueError(f"data must be a contiguous {dtype} tensor of {count} values")


def _stream_of(t):
    """The current stream's handle on t's device (what _stream_ptr returns, without its objects).

    The library launches on the current device, so t has to lie there.
    """
    device = t.get_device()
    if device != _current_device():
        raise ValueError(f"the tensors are on {t.device}, which is not the current device "
                         "(use torch.cuda.device)")
    return _raw_stream(device)


class MxFp4:
    """A matrix [rows, cols] (or ``batch`` of them) in MXFP4, as quantize_mxfp4 writes it.

    ``data`` is the device buffer (codes, then scales; imc.h has its layout), a
    contiguous uint8 tensor of at least mxfp4_bytes(batch, rows, cols) values;
    ``shape`` the shape of the values it stands for.
    """

    __slots__ = ("data", "batch", "rows", "cols", "batched")

    def __init__(self, data, batch, rows, cols, batched):
        torch = _torch or _setup()
        need = _size(batch, rows, cols)  # 0: empty, or no size at all
        if min(batch, rows, cols) < 0 or (need == 0 and batch * rows * cols):
            raise ValueError(f"no MXFP4 matrix has the sizes {batch}, {rows}, {cols}")
        if not batched and batch != 1:
            raise ValueError(f"{batch} matrices have to be batched")
        _check_buffer(data, torch.uint8, need)
        self._set(data, batch, rows, cols, batched)

    def _set(self, data, batch, rows, cols, batched):
        self.data, self.batch, self.rows, self.cols, self.batched = data, batch, rows, cols, batched
        return self

    @property
    def shape(self):
        return (self.batch, self.rows, self.cols) if self.batched else (self.rows, self.cols)

    @property
    def device(self):
        return self.data.device


def quantize_mxfp4(x, *, transpose=False):
    """x [rows, cols] or [batch, rows, cols] in MXFP4 (a scale for every 32 values of a row).

    x is float32, float16 or bfloat16, its rows may be strided.  ``transpose``
    quantises x^T instead (blocks down the columns of x), without a transposed
    copy: the operand of a product that sums over the rows of x.
    """
    batched = getattr(x, "ndim", 2) == 3
    if batched:
        dt, (batch, rows, cols), (step, ld, _) = _rows_of(x, "x", 3)
    else:
        dt, (rows, cols), (ld, _) = _rows_of(x, "x")
        batch, step = 1, 0
    r, c = (cols, rows) if transpose else (rows, cols)
    q = _torch.empty(_size(batch, r, c), dtype=_torch.uint8, device=x.device)
    rc = _calls.mxfp4_quantize(x.data_ptr(), dt, batch, rows, cols, step, ld,
                             1 if transpose else 0, q.data_ptr(), _stream_of(x))
    if rc:
        raise ImcError(rc, "mxfp4_quantize")
    return MxFp4.__new__(MxFp4)._set(q, batch, r, c, batched)


def dequantize_mxfp4(q, *, dtype=None):
    """The values an MxFp4 stands for, as a tensor of ``dtype`` (default float32)."""
    if not isinstance(q, MxFp4):
        raise TypeError("q must be an MxFp4")
    torch = _torch or _setup()  # q may have been loaded, and this be the first call
    dtype = torch.float32 if dtype is None else dtype
    dt, data = _dtype_id(dtype, "dtype"), q.data
    out = torch.empty(q.shape, dtype=dtype, device=data.device)
    rc = _calls.mxfp4_dequantize(data.data_ptr(), q.batch, q.rows, q.cols, dt, out.data_ptr(),
                               _stream_of(data))
    if rc:
        raise ImcError(rc, "mxfp4_dequantize")
    return out


def linear_mxfp4(x, w, bias=None, *, relu=False, out_dtype=None, out=None):
    """out = x @ w^T (+ bias) with both operands in MXFP4, summed in fp32.

    x [M, K] and w [N, K] are MxFp4, or float tensors that the call quantises
    (a weight that is used again is better quantised once, by quantize_mxfp4).
    bias [N] float32; ``relu`` fuses max(v, 0); out is [M, N] of ``out_dtype``
    (default: x's type, float32 for an MxFp4).
    """
    if isinstance(x, MxFp4):
        if x.batched:
            raise ValueError("x must be [M, K]")
        torch = _torch or _setup()
        like, dt, ld, M, K, default = x.data, MXFP4, 0, x.rows, x.cols, torch.float32
    else:
        dt, (M, K), (ld, _) = _rows_of(x, "x")
        like, default = x, x.dtype
    if not isinstance(w, MxFp4):
        _rows_of(w, "w")
        w = quantize_mxfp4(w)
    wd, N = w.data, w.rows
    if w.batched or w.cols != K:
        raise ValueError(f"w must be [N, K] = [N, {K}], got {list(w.shape)}")
    device = like.device
    if wd.device != device:
        raise ValueError("x and w must be on one device")
    if bias is not None:
        _check_plain(bias, "bias", _torch.float32, (N,), like)
    if out is None:
        out_dtype = default if out_dtype is None else out_dtype
        out = _torch.empty((M, N), dtype=out_dtype, device=device)
    else:
        out_dtype = out.dtype if out_dtype is None else out_dtype
        _check_plain(out, "out", out_dtype, (M, N), like)
    nbytes = _linear_size(M, K, dt)
    ws = _torch.empty(nbytes, dtype=_torch.uint8, device=device) if nbytes else None
    rc = _calls.mxfp4_linear(like.data_ptr(), dt, ld, wd.data_ptr(), _ptr(bias), out.data_ptr(),
                           _dtype_id(out_dtype, "out_dtype"), M, N, K, ACT_RELU if relu else 0,
                           _ptr(ws), nbytes, _stream_of(like))
    if rc:
        raise ImcError(rc, "mxfp4_linear")
    return out


def linear_mxfp4_backward(grad, x, w):
    """Gradients of ``linear_mxfp4(x, w)`` for grad [M, N], x [M, K], w [N, K].

    Returns (grad_x [M, K], grad_w [N, K]), each a 4-bit product whose operands
    are quantised along the axis that it sums over.  All tensors are contiguous
    and of one float type.  Without tokens (M = 0) or outputs (N = 0) both are 0.
    """
    dt, (M, N), _ = _rows_of(grad, "grad")
    K = _rows_of(x, "x")[1][1]
    dtype, device = grad.dtype, grad.device
    _check_plain(grad, "grad", dtype, (M, N), grad)
    _check_plain(x, "x", dtype, (M, K), grad)
    _check_plain(w, "w", dtype, (N, K), grad)
    if M == 0 or N == 0:
        return _torch.zeros_like(x), _torch.zeros_like(w)
    grad_x = _torch.empty((M, K), dtype=dtype, device=device)
    grad_w = _torch.empty((N, K), dtype=dtype, device=device)
    nbytes = _backward_size(M, N, K)
    ws = _torch.empty(nbytes, dtype=_torch.uint8, device=device)
    rc = _calls.mxfp4_linear_backward(grad.data_ptr(), x.data_ptr(), w.data_ptr(), dt, M, N, K,
                                    grad_x.data_ptr(), grad_w.data_ptr(), ws.data_ptr(), nbytes,
                                    _stream_of(grad))
    if rc:
        raise ImcError(rc, "mxfp4_linear_backward")
    return grad_x, grad_w


def route_experts(logits, k, bias=None, *, score="softmax", groups=1, top_groups=1,
                  renormalize=True, scale=1.0):
    """The k experts of each token and their weights, from router logits [T, E].

    Scores are softmax or sigmoid of the logits; the choice is by score + bias
    (bias [E] float32), within the ``top_groups`` best of ``groups`` equal runs of
    experts (a group counts by its two best); ties go to the lowest index.
    Returns (weights [T, k] float32, experts [T, k] int32), best first; the
    weights are the chosen scores, divided by their sum (``renormalize``), times
    ``scale``.
    """
    dt, (T, E), (ld, _) = _rows_of(logits, "logits")
    device = logits.device
    if bias is not None:
        _check_plain(bias, "bias", _torch.float32, (E,), logits)
    weights = _torch.empty((T, k), dtype=_torch.float32, device=device)
    experts = _torch.empty((T, k), dtype=_torch.int32, device=device)
    rc = _calls.moe_route(logits.data_ptr(), dt, T, E, ld, _ptr(bias), k, SCORES[score], groups,
                        top_groups, 1 if renormalize else 0, scale, weights.data_ptr(),
                        experts.data_ptr(), _stream_of(logits))
    if rc:
        raise ImcError(rc, "moe_route")
    return weights, experts


def route_experts_backward(grad_weights, logits, experts, *, score="softmax", renormalize=True,
                           scale=1.0):
    """Gradient of route_experts' weights with respect to the logits, [T, E] of their type."""
    dt, (T, E), (ld, _) = _rows_of(logits, "logits")
    k = experts.shape[-1]
    _check_plain(experts, "experts", _torch.int32, (T, k), logits)
    _check_plain(grad_weights, "grad_weights", _torch.float32, (T, k), logits)
    grad = _torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    rc = _calls.moe_route_backward(grad_weights.data_ptr(), logits.data_ptr(), dt, T, E, ld,
                                 experts.data_ptr(), k, SCORES[score], 1 if renormalize else 0,
                                 scale, grad.data_ptr(), _stream_of(logits))
    if rc:
        raise ImcError(rc, "moe_route_backward")
    return grad


class ExpertsLayout:
    """The slots (token * k + i) in expert order, as experts_layout writes them.

    ``offsets`` [E + 1]: where each expert's slots begin in ``order`` (slots of no
    expert come after offsets[E]); ``order`` [T * k].  ``data`` holds them and more
    (imc.h), at least moe_layout_size(T, k, E) int32 values.
    """

    __slots__ = ("data", "T", "k", "E")

    def __init__(self, data, T, k, E):
        torch = _torch or _setup()
        need = _layout_size(T, k, E)
        if need == 0:
            raise ValueError(f"no layout has the sizes {T}, {k}, {E}")
        _check_buffer(data, torch.int32, need)
        self._set(data, T, k, E)

    def _set(self, data, T, k, E):
        self.data, self.T, self.k, self.E = data, T, k, E
        return self

    @property
    def offsets(self):
        return self.data[: self.E + 1]

    @property
    def order(self):
        return self.data[2 * self.E + 3: 2 * self.E + 3 + self.T * self.k]


def experts_layout(experts, num_experts):
    """Sorts the slots of experts [T, k] int32 by expert (stable).

    An expert index outside [0, num_experts) leaves its slot out.
    """
    if not isinstance(experts, (_torch or _setup()).Tensor):
        raise TypeError("experts must be a torch.Tensor")
    if experts.dim() != 2:
        raise ValueError("experts must be [T, k]")
    T, k = experts.shape
    _check_plain(experts, "experts", _torch.int32, (T, k), experts)
    data = _torch.empty(_layout_size(T, k, num_experts), dtype=_torch.int32, device=experts.device)
    rc = _calls.moe_layout(experts.data_ptr(), T, k, num_experts, data.data_ptr(), _stream_of(experts))
    if rc:
        raise ImcError(rc, "moe_layout")
    return ExpertsLayout.__new__(ExpertsLayout)._set(data, T, k, num_experts)


def experts_linear_mxfp4(x, w, layout, bias=None, *, relu=False, out_dtype=None):
    """Each slot's row times its expert's weight: out[slot] = x[row] @ w[e]^T (+ bias[e]).

    x is [T, K] (every slot of a token takes its row) or [T * k, K] (a row for
    each slot); w an MxFp4 [E, N, K]; bias [E, N] float32; layout of
    experts_layout.  Returns [T * k, N] in slot order, of ``out_dtype`` (default:
    x's type); slots of no expert are 0.
    """
    dt, (rows, K), (ld, _) = _rows_of(x, "x")
    if not isinstance(w, MxFp4) or not w.batched:
        raise TypeError("w must be an MxFp4 [E, N, K]")
    if not isinstance(layout, ExpertsLayout):
        raise TypeError("layout must be an ExpertsLayout")
    T, k, E, N = layout.T, layout.k, layout.E, w.rows
    if w.batch != E or w.cols != K:
        raise ValueError(f"w must be [{E}, N, {K}], got {list(w.shape)}")
    if rows != T and rows != T * k:
        raise ValueError(f"x must have {T} or {T * k} rows, got {rows}")
    device, wd, ld_data = x.device, w.data, layout.data
    if wd.device != device or ld_data.device != device:
        raise ValueError("x, w and layout must be on one device")
    if bias is not None:
        _check_plain(bias, "bias", _torch.float32, (E, N), x)
    out_dtype = x.dtype if out_dtype is None else out_dtype
    out = _torch.empty((T * k, N), dtype=out_dtype, device=device)
    nbytes = _experts_size(T, k, E, K)
    ws = _torch.empty(nbytes, dtype=_torch.uint8, device=device) if nbytes else None
    rc = _calls.mxfp4_experts_linear(x.data_ptr(), dt, rows, ld, wd.data_ptr(), _ptr(bias),
                                   ld_data.data_ptr(), out.data_ptr(),
                                   _dtype_id(out_dtype, "out_dtype"), T, k, E, N, K,
                                   ACT_RELU if relu else 0, _ptr(ws), nbytes, _stream_of(x))
    if rc:
        raise ImcError(rc, "mxfp4_experts_linear")
    return out


def experts_linear_mxfp4_backward(grad, x, w, layout):
    """Gradients of ``experts_linear_mxfp4(x, quantize_mxfp4(w), layout)`` (without bias and ReLU).

    grad [T * k, N], x [T, K] or [T * k, K], w [E, N, K] are contiguous and of one
    float type.  Returns (grad_x of x's shape, grad_w [E, N, K]), 4-bit products whose
    operands are quantised along the axis that they sum over; a token's gradient is the
    fp32 sum over its slots, an expert without slots has a gradient of 0.
    """
    dt, (slots, N), _ = _rows_of(grad, "grad")
    if not isinstance(layout, ExpertsLayout):
        raise TypeError("layout must be an ExpertsLayout")
    T, k, E = layout.T, layout.k, layout.E
    _, (rows, K), _ = _rows_of(x, "x")
    dtype, device = grad.dtype, grad.device
    if rows != T and rows != T * k:
        raise ValueError(f"x must have {T} or {T * k} rows, got {rows}")
    _check_plain(grad, "grad", dtype, (T * k, N), grad)
    _check_plain(x, "x", dtype, (rows, K), grad)
    _check_plain(w, "w", dtype, (E, N, K), grad)
    if layout.data.device != device:
        raise ValueError("grad and layout must be on one device")
    if T == 0 or N == 0:
        return _torch.zeros_like(x), _torch.zeros_like(w)
    # A token's slots share its row: their products are summed in fp32 and rounded once
    # (4096 tokens, 8 of 64 experts, 1024 x 2048, bf16: 354 us, 341 with bf16 products).
    shared = rows != T * k
    grad_x = experts_linear_mxfp4(grad, quantize_mxfp4(w, transpose=True), layout,
                                  out_dtype=_torch.float32 if shared else dtype)
    if shared:
        slot_grads, grad_x = grad_x, _torch.empty((T, K), dtype=dtype, device=device)
        rc = _calls.moe_combine_f32(slot_grads.data_ptr(), None, T, k, K, grad_x.data_ptr(), dt,
                                    _stream_of(grad))
        if rc:
            raise ImcError(rc, "moe_combine_f32")
    grad_w = _torch.empty((E, N, K), dtype=dtype, device=device)
    nbytes = mxfp4_experts_weight_grad_workspace_bytes(T, k, E, N, K)
    ws = _torch.empty(nbytes, dtype=_torch.uint8, device=device)
    rc = _calls.mxfp4_experts_weight_grad(grad.data_ptr(), x.data_ptr(), dt, rows,
                                        layout.data.data_ptr(), grad_w.data_ptr(), T, k, E, N, K,
                                        ws.data_ptr(), nbytes, _stream_of(grad))
    if rc:
        raise ImcError(rc, "mxfp4_experts_weight_grad")
    return grad_x, grad_w


def _combine_dims(y, weights):
    dt, (rows, N), _ = _rows_of(y, "y")
    if not isinstance(weights, _torch.Tensor) or weights.dim() != 2:
        raise ValueError("weights must be a tensor [T, k]")
    T, k = weights.shape
    _check_plain(y, "y", y.dtype, (T * k, N), y)
    _check_plain(weights, "weights", _torch.float32, (T, k), y)
    return dt, T, k, N


def experts_combine(y, weights):
    """out[t] = sum_i weights[t, i] * y[t * k + i] for y [T * k, N], weights [T, k] float32."""
    dt, T, k, N = _combine_dims(y, weights)
    out = _torch.empty((T, N), dtype=y.dtype, device=y.device)
    rc = _calls.moe_combine(y.data_ptr(), dt, weights.data_ptr(), T, k, N, out.data_ptr(),
                          _stream_of(y))
    if rc:
        raise ImcError(rc, "moe_combine")
    return out


def experts_combine_backward(grad, y, weights):
    """Gradients of experts_combine for grad [T, N]: (grad_y [T * k, N], grad_weights [T, k])."""
    dt, T, k, N = _combine_dims(y, weights)
    _check_plain(grad, "grad", y.dtype, (T, N), y)
    grad_y = _torch.empty((T * k, N), dtype=y.dtype, device=y.device)
    grad_weights = _torch.empty((T, k), dtype=_torch.float32, device=y.device)
    rc = _calls.moe_combine_backward(grad.data_ptr(), y.data_ptr(), dt, weights.data_ptr(), T, k, N,
                                   grad_y.data_ptr(), grad_weights.data_ptr(), _stream_of(y))
    if rc:
        raise ImcError(rc, "moe_combine_backward")
    return grad_y, grad_weights


def _check_balance(logits, experts, score, offsets):
    dt, (T, E), (ld, _) = _rows_of(logits, "logits")
    if not isinstance(experts, _torch.Tensor) or experts.dim() != 2:
        raise ValueError("experts must be a tensor [T, k]")
    k, device = experts.shape[1], logits.get_device()
    _check_like(experts, "experts", _torch.int32, (T, k), device)
    S = 1
    if offsets is not None:
        if not isinstance(offsets, _torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 1:
            raise ValueError("offsets must be a tensor [S + 1]")
        S = offsets.shape[0] - 1
        _check_like(offsets, "offsets", _torch.int32, (S + 1,), device)
    return dt, T, E, ld, k, SCORES[score], S, device


def balance_loss(logits, experts, *, score="softmax", offsets=None):
    """How unevenly a router spreads its tokens over the experts, and the experts' counts.

    logits [T, E] and the experts [T, k] int32 that route_experts chose.  Sequence s holds
    the n tokens offsets[s] .. offsets[s + 1] (offsets [S + 1] int32, ascending; None: all
    tokens are one sequence); tokens of no sequence count nowhere.  Returns (loss [S]
    float32, counts [S, E] int32):

        loss[s] = E / (k n^2) * sum_e counts[s, e] * sum_t p[t, e]

    with p the softmax of the logits, or their sigmoids divided by their sum; 1 for an even
    choice, 0 for an empty sequence.  Scores are fp32; their sums are fp32 over 64 tokens and
    pairs of fp32 numbers (46 bits) beyond, in a fixed order.
    """
    dt, T, E, ld, k, score, S, _ = _check_balance(logits, experts, score, offsets)
    device = logits.device
    loss = _torch.empty((S,), dtype=_torch.float32, device=device)
    counts = experts.new_empty((S, E))  # (new_empty takes 0.3 us less than empty)
    nbytes = _balance_size(T, S, E)
    ws = experts.new_empty((nbytes >> 2,)) if nbytes else None
    rc = _calls.moe_balance(logits.data_ptr(), dt, T, E, ld, experts.data_ptr(), k, score,
                          _ptr(offsets), S, loss.data_ptr(), counts.data_ptr(), _ptr(ws), nbytes,
                          _stream_of(logits))
    if rc:
        raise ImcError(rc, "moe_balance")
    return loss, counts


def balance_loss_backward(grad_loss, logits, experts, counts, *, score="softmax", offsets=None,
                          grad_weights=None, renormalize=True, scale=1.0):
    """Gradient of balance_loss with respect to the logits, [T, E] of their type.

    grad_loss [S] float32, counts as balance_loss returned them (constant).  With
    grad_weights [T, k] float32 the gradient of route_experts' weights (of the same score,
    and this renormalize and scale) is added in the same pass: the sum of this and
    route_experts_backward, rounded once.  Tokens in no sequence have a gradient of 0 (of the
    weights' alone, if that is given), whatever their logits hold.
    """
    dt, T, E, ld, k, score, S, device = _check_balance(logits, experts, score, offsets)
    _check_like(grad_loss, "grad_loss", _torch.float32, (S,), device)
    _check_like(counts, "counts", _torch.int32, (S, E), device)
    if grad_weights is not None:
        _check_like(grad_weights, "grad_weights", _torch.float32, (T, k), device)
    grad = logits.new_empty((T, E))
    rc = _calls.moe_balance_backward(grad_loss.data_ptr(), logits.data_ptr(), dt, T, E, ld,
                                   experts.data_ptr(), k, score, counts.data_ptr(), _ptr(offsets), S,
                                   _ptr(grad_weights), 1 if renormalize else 0, scale,
                                   grad.data_ptr(), _stream_of(logits))
    if rc:
        raise ImcError(rc, "moe_balance_backward")
    return grad


def _check_like(t, name, dtype, shape, device):
    """_check_plain for the calls with many tensors: 0.35 us for 0.6."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on cuda:{device}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _check_adapters(x, a, b, layout, scale):
    dt, (T, K), (ld, _) = _rows_of(x, "x")
    if not isinstance(layout, ExpertsLayout):
        raise TypeError("layout must be an ExpertsLayout")
    if layout.k != 1 or layout.T != T:
        raise ValueError(f"layout must be of {T} rows with one adapter each")
    for t, name in ((a, "a"), (b, "b")):
        if not isinstance(t, _torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be a tensor of 3 dimensions")
    L, N, r = b.shape
    if layout.E != L:
        raise ValueError(f"layout must be of {L} adapters")
    dtype, device = x.dtype, x.get_device()
    _check_like(a, "a", dtype, (L, r, K), device)
    _check_like(b, "b", dtype, (L, N, r), device)
    if scale is not None:
        _check_like(scale, "scale", _torch.float32, (L,), device)
    if layout.data.get_device() != device:
        raise ValueError("x and layout must be on one device")
    return dt, T, L, r, K, N, ld, dtype, device


def adapters_linear(x, a, b, layout, base=None, *, scale=None, out=None):
    """Low-rank adapters of many requests: out[t] = base[t] + scale[l] * (x[t] @ a[l]^T) @ b[l]^T.

    x [T, K] (rows may be strided), a [L, r, K], b [L, N, r] and base [T, N], the shared
    projection's result (None: zeros), are of one float type; scale [L] float32 (None: ones).
    layout is experts_layout(which[:, None], L) for which [T] int32, row t's adapter l; a
    row whose number is outside [0, L) has none, and out[t] = base[t].  One layout serves
    every projection of a step.  Returns out [T, N]; ``out`` may be ``base`` (in place:
    rows without an adapter are left alone).  Sums are fp32 and the output is rounded once; in
    between x @ a^T is kept to 2^-17 of itself for the 16-bit types (two numbers of their size),
    to 2^-23 for float32, whose products are of three bf16 or TF32 parts with the smallest left out.
    """
    dt, T, L, r, K, N, ld, dtype, device = _check_adapters(x, a, b, layout, scale)
    if base is not None:
        _check_like(base, "base", dtype, (T, N), device)
    if out is None:
        out = x.new_empty((T, N)) if base is None else _torch.empty_like(base)
    else:
        _check_like(out, "out", dtype, (T, N), device)
    nbytes = _lowrank_size(T, L, r)
    ws = layout.data.new_empty((nbytes >> 2,)) if nbytes else None
    rc = _calls.lowrank_linear(x.data_ptr(), dt, ld, a.data_ptr(), b.data_ptr(), _ptr(scale),
                             layout.data.data_ptr(), _ptr(base), out.data_ptr(), T, L, r, K, N,
                             _ptr(ws), nbytes, _stream_of(x))
    if rc:
        raise ImcError(rc, "lowrank_linear")
    return out


def adapters_linear_backward(grad, x, a, b, layout, base=None, *, scale=None):
    """Gradients of ``adapters_linear(x, a, b, layout, scale=scale)`` for grad [T, N].

    Returns (grad_x [T, K], grad_a [L, r, K], grad_b [L, N, r]).  base [T, K] is added to
    grad_x (the gradient through the shared projection).  All tensors are contiguous and
    of one float type; an adapter without rows has gradients of 0.  grad @ b and x @ a^T are
    kept as in adapters_linear (float16 in the weights' gradients: as two bfloat16 numbers).
    """
    dt, T, L, r, K, N, _, dtype, device = _check_adapters(x, a, b, layout, scale)
    _check_like(x, "x", dtype, (T, K), device)
    _check_like(grad, "grad", dtype, (T, N), device)
    if base is not None:
        _check_like(base, "base", dtype, (T, K), device)
    if T == 0 or N == 0:
        grad_x = _torch.zeros_like(x) if base is None else base.clone()
        return grad_x, _torch.zeros_like(a), _torch.zeros_like(b)
    grad_x, grad_a, grad_b = _torch.empty_like(x), _torch.empty_like(a), _torch.empty_like(b)
    nbytes = _lowrank_back_size(T, r)
    ws = layout.data.new_empty((nbytes >> 2,))
    rc = _calls.lowrank_linear_backward(grad.data_ptr(), x.data_ptr(), a.data_ptr(), b.data_ptr(), dt,
                                      _ptr(scale), layout.data.data_ptr(), _ptr(base),
                                      grad_x.data_ptr(), grad_a.data_ptr(), grad_b.data_ptr(), T, L,
                                      r, K, N, ws.data_ptr(), nbytes, _stream_of(x))
    if rc:
        raise ImcError(rc, "lowrank_linear_backward")
    return grad_x, grad_a, grad_b
