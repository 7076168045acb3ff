"""What the torch-level 4-bit and expert functions check before anything is launched,
and how they start up.  No GPU: tensors stand in for CUDA ones where a check needs one,
and no call gets as far as a launch."""
import os
import subprocess
import sys

import pytest
import torch

from addmm_implicit_im2col_gb300 import binding, build
from conftest import ROOT


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def fresh(code):
    """Runs code in a new process that sees no GPU; it has to exit with 0."""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES=""), timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("call", ["binding.dequantize_mxfp4(q)", "binding.linear_mxfp4(q, q)"])
def test_a_stored_matrix_may_come_first(call):
    """An MxFp4 made from a stored buffer, before any other call of the process: the call
    sets the module up and fails for want of a GPU alone."""
    fresh(f"""
import torch
from addmm_implicit_im2col_gb300 import binding
data = torch.zeros(binding.mxfp4_bytes(1, 4, 64), dtype=torch.uint8)
q = binding.MxFp4(data, 1, 4, 64, False)
try:
    {call}
except (RuntimeError, ValueError):  # no GPU: from torch or the library
    pass
""")


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The library launches on the current device: a tensor of another one (or of the host)
    may not get its stream."""
    class Tensor:
        def __init__(self, device):
            self.device, self.get_device = f"cuda:{device}", lambda: device

    binding._setup()
    monkeypatch.setattr(binding, "_current_device", lambda: 1, raising=False)
    monkeypatch.setattr(binding, "_raw_stream", lambda device: 100 + device)
    assert binding._stream_of(Tensor(1)) == 101
    for device in (0, 2, -1):
        with pytest.raises(ValueError, match="current device"):
            binding._stream_of(Tensor(device))


def test_a_matrix_needs_the_buffer_of_its_size():
    """The kernels read as far as the shape says, so a buffer that is too short, of another
    type or not contiguous is refused when the matrix is made."""
    def make(data, batch=1, rows=150, cols=300, batched=False):
        return binding.MxFp4(data, batch, rows, cols, batched)

    need = binding.mxfp4_bytes(1, 150, 300)
    good = torch.zeros(need, dtype=torch.uint8)
    assert make(good).shape == (150, 300) and make(good).data is good
    assert make(torch.zeros(need + 1, dtype=torch.uint8)).shape == (150, 300)
    assert make(torch.zeros(binding.mxfp4_bytes(3, 150, 300), dtype=torch.uint8), 3, batched=True).shape == (3, 150, 300)
    assert make(torch.zeros(0, dtype=torch.uint8), rows=0).shape == (0, 300)
    with pytest.raises(TypeError):
        make(bytes(need))
    for data in (good[:-1], good.view(torch.int8), good.float(), good.view(2, -1),
                 torch.zeros(2 * need, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            make(data)
    for batch, rows, cols, batched in ((2, 150, 300, True), (1, 151, 300, False), (1, 150, 321, False),
                                       (1, -1, 300, False), (1, 150, -300, False), (-1, -150, 300, True),
                                       (1, 2 ** 31, 300, False), (1, 2 ** 30, 2 ** 30, False)):
        with pytest.raises(ValueError):
            make(good, batch, rows, cols, batched)
    with pytest.raises(ValueError):  # two matrices that say they are one
        make(torch.zeros(binding.mxfp4_bytes(2, 150, 300), dtype=torch.uint8), 2, batched=False)


def test_a_layout_needs_the_buffer_of_its_size():
    def make(data, T=70, k=3, E=5):
        return binding.ExpertsLayout(data, T, k, E)

    need = binding.moe_layout_size(70, 3, 5)
    good = torch.zeros(need, dtype=torch.int32)
    made = make(good)
    assert made.data is good and made.offsets.numel() == 6 and made.order.numel() == 210
    assert make(torch.zeros(need + 4, dtype=torch.int32)).T == 70
    assert make(torch.zeros(binding.moe_layout_size(0, 3, 5), dtype=torch.int32), T=0).order.numel() == 0
    with pytest.raises(TypeError):
        make([0] * need)
    for data in (good[:-1], good.long(), good.view(torch.float32), torch.zeros(2 * need, dtype=torch.int32)[::2],
                 good[: need // 2 * 2].view(2, -1)):
        with pytest.raises(ValueError):
            make(data)
    for T, k, E in ((71, 3, 5), (70, 4, 5), (70, 3, 6), (-1, 3, 5), (70, 0, 5), (70, 33, 5), (70, 3, 1025), (70, 3, 0)):
        with pytest.raises(ValueError):
            make(good, T, k, E)


def test_layout_refuses_places_that_pass_32_bits():
    """A slot's last place among the runs of experts, filled up to 128 rows and those in tiles
    of 224, is held in 32 bits."""
    P1, P2 = 0x100000000, 0x10000000000
    for E in (1, 7, 1024):
        rows = (2 ** 31 - 1) // 224 * 128  # the largest number of filled-up rows
        most = rows - 127 * E              # slots that may need as many
        assert binding.moe_layout_size(most, 1, E) > 0
        for T, k in ((most + 1, 1), (most // 3 + 1, 3), (2 ** 31 - 2, 1)):
            assert binding.moe_layout_size(T, k, E) == 0
            assert binding.moe_layout(P1, T, k, E, P2, None) == binding.IMC_ERR_SHAPE
            assert binding.mxfp4_experts_linear_workspace_bytes(T, k, E, 64) == 0
            assert binding.mxfp4_experts_weight_grad_workspace_bytes(T, k, E, 64, 64) == 0


class OnGpu(torch.Tensor):
    """A tensor of the host that passes for a CUDA one."""
    is_cuda = True


def on_gpu(*shape, dtype=torch.float32):
    return torch.ones(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N", [(0, 70), (5, 0), (0, 0)])
def test_gradients_of_an_empty_product(M, N, dtype):
    """A product without tokens or without outputs has gradients of 0, and nothing to launch."""
    dx, dw = binding.linear_mxfp4_backward(on_gpu(M, N, dtype=dtype), on_gpu(M, 64, dtype=dtype),
                                           on_gpu(N, 64, dtype=dtype))
    assert dx.shape == (M, 64) and dw.shape == (N, 64) and dx.dtype == dw.dtype == dtype
    assert bool((dx == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("T,N,per_slot", [(0, 20, False), (6, 0, False), (6, 0, True), (0, 0, True)])
def test_gradients_of_an_empty_product_of_experts(T, N, per_slot):
    layout = binding.ExpertsLayout(torch.zeros(binding.moe_layout_size(T, 2, 4), dtype=torch.int32), T, 2, 4)
    x = on_gpu(2 * T if per_slot else T, 64)
    dx, dw = binding.experts_linear_mxfp4_backward(on_gpu(2 * T, N), x, on_gpu(4, N, 64), layout)
    assert dx.shape == x.shape and dw.shape == (4, N, 64)
    assert bool((dx == 0).all()) and bool((dw == 0).all())


def test_sum_of_fp32_rows_checks_its_arguments():
    def call(y=0x100000000, w=0x200000000, T=4, k=2, N=8, out=0x300000000, dtype=binding.BF16):
        return binding.moe_combine_f32(y, w, T, k, N, out, dtype, None)

    assert call(dtype=3) == call(dtype=-1) == binding.IMC_ERR_ARG
    assert call(y=0x100000002) == call(out=0x300000001) == call(w=0x200000001) == binding.IMC_ERR_ARG
    assert call(dtype=binding.F32, out=0x300000002) == binding.IMC_ERR_ARG
    assert call(T=-1) == call(k=0) == call(k=33) == call(N=2 ** 31) == binding.IMC_ERR_SHAPE
    assert call(y=None) == call(out=None) == binding.IMC_ERR_NULL
    assert call(out=0x100000000 + 4 * 2 * 8 * 4 - 2) == call(out=0x200000000) == binding.IMC_ERR_ALIAS
    assert call(T=0) == call(N=0) == binding.IMC_OK
    binding._setup()
    assert binding._calls.moe_combine_f32(1, 0, 4, 2, 8, 0x300000000, 2, None) == binding.IMC_ERR_ARG
    with pytest.raises(TypeError):
        binding._calls.moe_combine_f32(0x100000000, 0, 4, 2, 8, 0x300000000, 2)


def test_without_the_python_module_the_calls_go_through_ctypes():
    """Where the module over the entry points was not built, the same entry points are called
    through ctypes: the same names, arguments and statuses."""
    fresh("""
import sys
sys.modules["addmm_implicit_im2col_gb300._calls"] = None  # as if it were not there
import torch
from addmm_implicit_im2col_gb300 import binding
binding._setup()
calls = binding._calls
for name in ("mxfp4_quantize", "mxfp4_dequantize", "mxfp4_linear", "mxfp4_linear_backward", "moe_route",
             "moe_route_backward", "moe_layout", "mxfp4_experts_linear", "mxfp4_experts_weight_grad",
             "moe_combine", "moe_combine_f32", "moe_combine_backward"):
    zeros = [0.0 if t is binding._dbl else 0 for t in binding.SIGNATURES[name][1]]
    assert getattr(calls, name)(*zeros) == getattr(binding.load(), name)(*zeros), name
P1, P2 = 0x100000000, 0x200000000
assert calls.mxfp4_quantize(P1, 99, 1, 8, 64, 0, 64, 0, P2, None) == binding.IMC_ERR_ARG
assert calls.mxfp4_quantize(None, 0, 1, 8, 64, 0, 64, 0, P2, None) == binding.IMC_ERR_NULL
assert calls.mxfp4_quantize(P1, 0, 1, 8, 64, 0, 64, 0, P1, 0) == binding.IMC_ERR_ALIAS
""")


def test_build_without_python_headers(monkeypatch, tmp_path, capfd):
    """The C library does not need them: its build goes through, without the module."""
    monkeypatch.setattr(build, "CALLS_PATH", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.build() == build.LIB_PATH
    assert not (tmp_path / "_calls.so").exists() and "Python.h" in capfd.readouterr().err


def test_the_module_is_built_for_this_python():
    """Its name holds the interpreter's version: another one does not take it for its own."""
    import sysconfig
    assert os.path.basename(build.CALLS_PATH) == "_calls" + sysconfig.get_config_var("EXT_SUFFIX")
    binding._setup()
    assert binding._calls.__file__ == build.CALLS_PATH
