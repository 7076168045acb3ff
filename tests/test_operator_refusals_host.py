"""Refusals of the 4-bit and expert entry points: every bad argument gets its
documented status before any CUDA call (fake, never dereferenced addresses), a
well-formed call without a GPU fails loudly, and the torch-level functions check
types, shapes and devices."""
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding, build
from test_boundary_host import without_gpu

P1, P2, P3, P4, P5 = (0x100000000 * i for i in range(1, 6))
ARG, SHAPE, NULL, ALIAS = (binding.IMC_ERR_ARG, binding.IMC_ERR_SHAPE, binding.IMC_ERR_NULL,
                           binding.IMC_ERR_ALIAS)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def quantize(x=P1, dtype=0, batch=1, rows=8, cols=64, batch_stride=0, row_stride=64, transpose=0,
             q=P2):
    return binding.mxfp4_quantize(x, dtype, batch, rows, cols, batch_stride, row_stride, transpose,
                                  q, None)


def dequantize(q=P1, batch=1, rows=8, cols=64, dtype=0, out=P2):
    return binding.mxfp4_dequantize(q, batch, rows, cols, dtype, out, None)


def linear(x=P1, x_dtype=0, row_stride=64, w=P2, bias=P3, out=P4, out_dtype=0, M=9, N=8, K=64,
           flags=0, ws=P5, nbytes=1 << 20):
    return binding.mxfp4_linear(x, x_dtype, row_stride, w, bias, out, out_dtype, M, N, K, flags, ws,
                                nbytes, None)


def backward(grad=P1, x=P2, w=P3, dtype=0, M=8, N=8, K=64, gx=P4, gw=P5, ws=None, nbytes=0):
    return binding.mxfp4_linear_backward(grad, x, w, dtype, M, N, K, gx, gw, ws, nbytes, None)


def route(logits=P1, dtype=0, T=4, E=16, row_stride=16, bias=P2, k=2, score=0, groups=1, top=1,
          renorm=1, scale=1.0, weights=P3, experts=P4):
    return binding.moe_route(logits, dtype, T, E, row_stride, bias, k, score, groups, top, renorm,
                             scale, weights, experts, None)


def route_backward(g=P1, logits=P2, dtype=0, T=4, E=16, row_stride=16, experts=P3, k=2, score=0,
                   renorm=1, scale=1.0, out=P4):
    return binding.moe_route_backward(g, logits, dtype, T, E, row_stride, experts, k, score, renorm,
                                      scale, out, None)


def experts_linear(x=P1, x_dtype=0, rows=400, row_stride=64, w=P2, bias=None, layout=P3, out=P4,
                   out_dtype=0, T=400, k=2, E=16, N=8, K=64, flags=0, ws=P5, nbytes=1 << 22):
    return binding.mxfp4_experts_linear(x, x_dtype, rows, row_stride, w, bias, layout, out,
                                        out_dtype, T, k, E, N, K, flags, ws, nbytes, None)


def weight_grad(grad=P1, x=P2, dtype=0, rows=4, layout=P3, gw=P4, T=4, k=2, E=16, N=8, K=64, ws=P5,
                nbytes=1 << 22):
    return binding.mxfp4_experts_weight_grad(grad, x, dtype, rows, layout, gw, T, k, E, N, K, ws,
                                             nbytes, None)


def combine(y=P1, dtype=0, w=P2, T=4, k=2, N=8, out=P3):
    return binding.moe_combine(y, dtype, w, T, k, N, out, None)


def combine_backward(grad=P1, y=P2, dtype=0, w=P3, T=4, k=2, N=8, gy=P4, gw=P5):
    return binding.moe_combine_backward(grad, y, dtype, w, T, k, N, gy, gw, None)


BAD = [
    (quantize, dict(dtype=3), ARG), (quantize, dict(dtype=-1), ARG), (quantize, dict(transpose=2), ARG),
    (quantize, dict(rows=-1), SHAPE), (quantize, dict(cols=2 ** 31), SHAPE),
    (quantize, dict(row_stride=63), SHAPE), (quantize, dict(batch_stride=-1), SHAPE),
    (quantize, dict(x=None), NULL), (quantize, dict(q=None), NULL), (quantize, dict(q=P2 + 8), ARG),
    (quantize, dict(x=P1 + 2), ARG), (quantize, dict(q=P1 + 16), ALIAS),
    (dequantize, dict(dtype=3), ARG), (dequantize, dict(rows=-1), SHAPE), (dequantize, dict(q=None), NULL),
    (dequantize, dict(out=None), NULL), (dequantize, dict(q=P1 + 4), ARG), (dequantize, dict(out=P1), ALIAS),
    (linear, dict(x_dtype=4), ARG), (linear, dict(out_dtype=3), ARG), (linear, dict(flags=1), ARG),
    (linear, dict(M=-1), SHAPE), (linear, dict(K=0), SHAPE), (linear, dict(N=2 ** 31), SHAPE),
    (linear, dict(row_stride=8), SHAPE), (linear, dict(x=None), NULL), (linear, dict(w=None), NULL),
    (linear, dict(out=None), NULL), (linear, dict(w=P2 + 1), ARG), (linear, dict(out=P4 + 2), ARG),
    (linear, dict(x_dtype=3, x=P1 + 8), ARG), (linear, dict(nbytes=16), ARG), (linear, dict(ws=P5 + 4), ARG),
    (linear, dict(out=P1), ALIAS), (linear, dict(out=P2), ALIAS), (linear, dict(out=P3), ALIAS),
    (linear, dict(ws=P4), ALIAS), (linear, dict(ws=P1), ALIAS), (linear, dict(ws=P2), ALIAS),
    (backward, dict(dtype=3), ARG), (backward, dict(M=0), SHAPE), (backward, dict(K=-1), SHAPE),
    (backward, dict(grad=None), NULL), (backward, dict(w=None), NULL), (backward, dict(x=None), NULL),
    (backward, dict(gx=P1), ALIAS), (backward, dict(gw=P2), ALIAS), (backward, dict(gw=P4), ALIAS),
    (backward, dict(gx=P4 + 2), ARG), (backward, dict(ws=0x900000000, nbytes=8), ARG),
    (route, dict(dtype=3), ARG), (route, dict(score=2), ARG), (route, dict(renorm=2), ARG),
    (route, dict(scale=float("nan")), ARG), (route, dict(T=-1), SHAPE), (route, dict(E=0), SHAPE),
    (route, dict(E=1025, row_stride=2000), SHAPE), (route, dict(k=0), SHAPE), (route, dict(k=17), SHAPE),
    (route, dict(E=64, row_stride=64, k=33), SHAPE), (route, dict(groups=3), SHAPE),
    (route, dict(groups=4, top=5), SHAPE), (route, dict(groups=4, top=0), SHAPE),
    (route, dict(groups=16, top=1), SHAPE), (route, dict(row_stride=15), SHAPE),
    (route, dict(logits=None), NULL), (route, dict(weights=None), NULL), (route, dict(experts=None), NULL),
    (route, dict(weights=P1), ALIAS), (route, dict(experts=P3), ALIAS), (route, dict(weights=P3 + 2), ARG),
    (route_backward, dict(dtype=9), ARG), (route_backward, dict(E=0), SHAPE), (route_backward, dict(g=None), NULL),
    (route_backward, dict(out=None), NULL), (route_backward, dict(out=P2), ALIAS),
    (experts_linear, dict(x_dtype=3), ARG), (experts_linear, dict(flags=2), ARG),
    (experts_linear, dict(rows=401), SHAPE), (experts_linear, dict(E=0), SHAPE), (experts_linear, dict(k=33), SHAPE),
    (experts_linear, dict(K=0), SHAPE), (experts_linear, dict(layout=None), NULL),
    (experts_linear, dict(w=None), NULL), (experts_linear, dict(nbytes=100), ARG),
    (experts_linear, dict(out=P1), ALIAS), (experts_linear, dict(out=P3), ALIAS), (experts_linear, dict(ws=P4), ALIAS),
    (combine, dict(dtype=3), ARG), (combine, dict(k=0), SHAPE), (combine, dict(y=None), NULL),
    (combine, dict(out=P1), ALIAS), (combine, dict(out=None), NULL),
    (weight_grad, dict(dtype=3), ARG), (weight_grad, dict(rows=5), SHAPE), (weight_grad, dict(T=0), SHAPE),
    (weight_grad, dict(N=0), SHAPE), (weight_grad, dict(x=None), NULL), (weight_grad, dict(layout=None), NULL),
    (weight_grad, dict(nbytes=64), ARG), (weight_grad, dict(gw=P1), ALIAS), (weight_grad, dict(ws=P4), ALIAS),
    (combine_backward, dict(dtype=3), ARG), (combine_backward, dict(T=-1), SHAPE),
    (combine_backward, dict(gy=None), NULL), (combine_backward, dict(gy=P2), ALIAS),
    (combine_backward, dict(gw=P4), ALIAS),
]


@pytest.mark.parametrize("call,args,want", BAD, ids=lambda v: getattr(v, "__name__", None) or str(v))
def test_refused(call, args, want):
    assert call(**args) == want


def test_layout_refusals():
    assert binding.moe_layout(P1, 4, 2, 0, P2, None) == SHAPE
    assert binding.moe_layout(P1, 4, 33, 8, P2, None) == SHAPE
    assert binding.moe_layout(P1, 2 ** 30, 4, 8, P2, None) == SHAPE
    assert binding.moe_layout(None, 4, 2, 8, P2, None) == NULL
    assert binding.moe_layout(P1, 4, 2, 8, None, None) == NULL
    assert binding.moe_layout(P1, 4, 2, 8, P1 + 4, None) == ALIAS
    assert binding.moe_layout(P1, 4, 2, 8, P2 + 2, None) == ARG


def test_sizes():
    # codes, up to 512 bytes, then scale atoms of 128 rows x 4 blocks
    assert binding.mxfp4_bytes(1, 1, 1) == 512 + 512
    assert binding.mxfp4_bytes(2, 129, 129) == -(-2 * 129 * 80 // 512) * 512 + 2 * 2 * 2 * 512
    assert binding.mxfp4_bytes(1, -1, 4) == 0 and binding.mxfp4_bytes(1, 2 ** 31 - 1, 2 ** 31 - 1) == 0
    assert binding.mxfp4_linear_workspace_bytes(9, 64, 0) == binding.mxfp4_bytes(1, 9, 64)
    assert binding.mxfp4_linear_workspace_bytes(8, 64, 0) == 0  # quantised within the product
    assert binding.mxfp4_linear_workspace_bytes(8, 64, binding.MXFP4) == 0
    assert binding.moe_layout_size(4, 2, 8) == 2 * 8 + 3 + 24
    assert binding.mxfp4_experts_linear_workspace_bytes(4, 33, 8, 64) == 0


def test_empty_calls_do_nothing():
    assert quantize(rows=0) == 0 and dequantize(cols=0) == 0 and linear(M=0) == 0 and linear(N=0) == 0
    assert route(T=0) == 0 and route_backward(T=0) == 0 and combine(T=0) == 0 and combine(N=0) == 0
    assert experts_linear(T=0, rows=0) == 0 and backward(gx=None, gw=None) == 0
    assert binding.last_kernel() == "none"


def test_without_a_gpu_calls_fail_loudly():
    calls = [("mxfp4_quantize", [P1, 0, 1, 8, 64, 0, 64, 0, P2, None]),
             ("mxfp4_dequantize", [P1, 1, 8, 64, 0, P2, None]),
             ("mxfp4_linear", [P1, 0, 64, P2, None, P4, 0, 8, 8, 64, 0, P5, 1 << 20, None]),
             ("mxfp4_linear_backward", [P1, P2, P3, 0, 8, 8, 64, P4, P5, None, 0, None]),
             ("moe_route", [P1, 0, 4, 16, 16, None, 2, 0, 1, 1, 1, 1.0, P3, P4, None]),
             ("moe_route_backward", [P1, P2, 0, 4, 16, 16, P3, 2, 0, 1, 1.0, P4, None]),
             ("moe_layout", [P1, 4, 2, 8, P2, None]),
             ("mxfp4_experts_linear", [P1, 0, 4, 64, P2, None, P3, P4, 0, 4, 2, 16, 8, 64, 0, P5, 1 << 22, None]),
             ("mxfp4_experts_weight_grad", [P1, P2, 0, 4, P3, P4, 4, 2, 16, 8, 64, P5, 1 << 22, None]),
             ("moe_combine", [P1, 0, P2, 4, 2, 8, P3, None]),
             ("moe_combine_backward", [P1, P2, 0, P3, 4, 2, 8, P4, P5, None])]
    assert without_gpu(calls) == [binding.IMC_ERR_DEVICE] * len(calls)


def test_torch_level_checks():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        binding.quantize_mxfp4(x)  # not on the GPU
    with pytest.raises(TypeError):
        binding.quantize_mxfp4([1.0])
    with pytest.raises(ValueError):
        binding.linear_mxfp4(x, x)
    with pytest.raises(TypeError):
        binding.dequantize_mxfp4(x)
    with pytest.raises(ValueError):
        binding.route_experts(x, 2)
    with pytest.raises(ValueError):
        binding.experts_layout(x.int(), 4)
    with pytest.raises(TypeError):
        binding.experts_layout([0], 4)
    with pytest.raises(ValueError):
        binding.experts_combine(x, x)
    with pytest.raises(ValueError):
        binding.linear_mxfp4_backward(x, x, x)
    with pytest.raises(ValueError):
        binding.experts_linear_mxfp4(x, None, None)


def test_python_module_calls_the_same_entry_points():
    """The module that the torch-level functions call: statuses, counts and types of arguments."""
    binding._setup()
    calls = binding._calls
    assert calls.mxfp4_quantize(P1, 99, 1, 8, 64, 0, 64, 0, P2, None) == ARG
    assert calls.mxfp4_quantize(P1, 0, 1, 8, 64, 0, 63, 0, P2, 0) == SHAPE
    assert calls.mxfp4_quantize(None, 0, 1, 8, 64, 0, 64, 0, P2, None) == NULL
    assert calls.mxfp4_quantize(P1, 0, 1, 8, 64, 0, 64, 0, P1, None) == ALIAS
    for name in ("mxfp4_quantize", "mxfp4_dequantize", "mxfp4_linear", "mxfp4_linear_backward",
                 "moe_route", "moe_route_backward", "moe_layout", "mxfp4_experts_linear",
                 "mxfp4_experts_weight_grad", "moe_combine", "moe_combine_backward"):
        args = binding.SIGNATURES[name][1]
        zeros = [0.0 if t is binding._dbl else 0 for t in args]
        assert getattr(calls, name)(*zeros) == getattr(binding.load(), name)(*zeros), name
        with pytest.raises(TypeError, match=name):
            getattr(calls, name)(*zeros[1:])
        with pytest.raises(TypeError):
            getattr(calls, name)("x", *zeros[1:])
    with pytest.raises(OverflowError):
        calls.mxfp4_quantize(P1, 1 << 40, 1, 8, 64, 0, 64, 0, P2, None)
    with pytest.raises(OverflowError):
        calls.mxfp4_quantize(P1, 0, 1 << 80, 8, 64, 0, 64, 0, P2, None)
