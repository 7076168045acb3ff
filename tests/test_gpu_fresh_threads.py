"""Every operator as the first CUDA work of a host thread.

Such a thread has no current context until a runtime call binds one, and encoding a tensor map
needs it.  Results are those of the same call in the main thread; the outputs of that one are
free again, so that the thread's allocations need no CUDA call either.
"""
import threading

import pytest
import torch

from addmm_implicit_im2col_gb300 import binding

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def normal(*shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(sum(shape))
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def fp32(mode):
    x, w, s = normal(256, 320), normal(384, 320), normal(384)
    img, filt = normal(2, 16, 24, 24), normal(64, 16, 3, 3)
    return {f"addmm {mode}": lambda: binding.addmm(s, x, w.t().contiguous(), mode=mode),
            f"linear {mode}": lambda: binding.linear(x, w, mode=mode),
            f"conv2d {mode}": lambda: binding.conv2d(img, filt, padding=1, mode=mode),
            f"conv2d 7x7 {mode}": lambda: binding.conv2d(img[:, :3].contiguous(), filt[:, :3].contiguous(), mode=mode)}


def products():
    w = binding.quantize_mxfp4(normal(512, 256, dtype=torch.bfloat16))
    x, few = normal(300, 256, dtype=torch.bfloat16), normal(3, 256, dtype=torch.bfloat16)
    xq, grad, wide = binding.quantize_mxfp4(x), normal(300, 512, dtype=torch.bfloat16), normal(512, 256, dtype=torch.bfloat16)
    we = binding.quantize_mxfp4(normal(4, 512, 256, dtype=torch.bfloat16))
    experts = (torch.arange(600).view(300, 2) % 4).int().cuda()
    layout = binding.experts_layout(experts, 4)
    return {"mxfp4 quantise": lambda: binding.quantize_mxfp4(x).data,
            "mxfp4 linear": lambda: binding.linear_mxfp4(x, w),
            "mxfp4 linear of mxfp4": lambda: binding.linear_mxfp4(xq, w),
            "mxfp4 linear of few": lambda: binding.linear_mxfp4(few, w),
            "mxfp4 gradients": lambda: binding.linear_mxfp4_backward(grad, x, wide),
            "experts layout": lambda: binding.experts_layout(experts, 4).data[:6],
            "experts": lambda: binding.experts_linear_mxfp4(x, we, layout),
            "route": lambda: binding.route_experts(x, 2)}


def adapters(name, T, L, r, K, N):
    dtype = DTYPES[name]
    x, a, b = normal(T, K, dtype=dtype), normal(L, r, K, dtype=dtype), normal(L, N, r, dtype=dtype)
    grad = normal(T, N, dtype=dtype)
    layout = binding.experts_layout((torch.arange(T) % L)[:, None].int().contiguous().cuda(), L)
    label = f"{name} {T} of {L}"
    return {f"adapters {label}": lambda: binding.adapters_linear(x, a, b, layout),
            f"adapters' gradients {label}": lambda: binding.adapters_linear_backward(grad, x, a, b, layout)}


def balance(T):
    x = normal(T, 64)
    experts = x.topk(2, -1).indices.int().contiguous()
    loss, counts = binding.balance_loss(x, experts)
    return {f"balance loss {T}": lambda: binding.balance_loss(x, experts),
            f"balance gradient {T}": lambda: binding.balance_loss_backward(loss, x, experts, counts)}


GROUPS = {**{f"fp32 {m}": (lambda m=m: fp32(m)) for m in ("default", "tf32", "simt", "force_tc3", "force_tc1", "direct")},
          "products": products,
          **{f"adapters {n} {T}": (lambda n=n, T=T, L=L: adapters(n, T, L, 16, 256, 384))
             for n in DTYPES for T, L in ((5, 3), (3000, 2))},
          "balance 40": lambda: balance(40), "balance 2000": lambda: balance(2000)}


@pytest.mark.parametrize("group", GROUPS)
def test_first_call_of_a_thread(group):
    for name, call in GROUPS[group]().items():
        if name.startswith(("addmm", "linear")) and group.endswith("direct"):
            continue  # a mode of conv2d alone
        want = call()
        want = [t.cpu() for t in (want if isinstance(want, tuple) else (want,))]
        got = []

        def work():
            try:
                got.append(call())
            except Exception as error:
                got.append(error)

        thread = threading.Thread(target=work)
        thread.start()
        thread.join()
        assert not isinstance(got[0], Exception), f"{name}: {got[0]}"
        result = got[0] if isinstance(got[0], tuple) else (got[0],)
        assert all(torch.equal(p, q.cpu()) for p, q in zip(want, result)), name


def test_capture_in_a_thread():
    """The first call of a thread within a capture (the device has seen the call before)."""
    calls = [call for group in ("adapters bf16 3000", "adapters f32 5", "products") for name, call in GROUPS[group]().items()
             if name != "mxfp4 quantise"]  # (a buffer has bytes between its rows that no call writes)
    want = [c() for c in calls]
    got = []

    def work():
        try:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs = [c() for c in calls]
            graph.replay()
            torch.cuda.synchronize()
            got.append(outs)
        except Exception as error:
            got.append(error)

    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    assert isinstance(got[0], list), got[0]
    for p, q in zip(want, got[0]):
        p, q = (t if isinstance(t, tuple) else (t,) for t in (p, q))
        assert all(torch.equal(u, v) for u, v in zip(p, q))
