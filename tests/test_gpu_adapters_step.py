"""Adapters, router and balance loss together, as a training step and a serving step use them.

Training, in fp32: y = x W^T (linear), out = y + adapters, logits = out R^T (linear), the
routing weights and the balance loss of the sequences; all gradients against those of the
same step in 64 bits with the same choice of experts.  A product of the step is off by at most
1e-5 of sum |x w| (the linear's and the adapters' bounds), which for these random values and
256 terms is about ten times its size; scores, weights and loss add some roundings (1e-6).
Errors of five products one after the other stay below 5 * 1e-4 of the result's norm: 1e-3.
"""
import numpy as np
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding
from test_gpu_adapters import Case, within

pytestmark = pytest.mark.gpu


class Step:
    """One layer: a frozen projection with adapters, whose outputs a router sees."""

    def __init__(self, T, L, r, K, N, E, k, lengths, score, seed=0):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, size=1.0):
            return (size * torch.randn(*shape, generator=g)).cuda()

        self.L, self.k, self.score = L, k, score
        self.x, self.w, self.router = normal(T, K), normal(N, K, size=K ** -0.5), normal(E, N, size=N ** -0.5)
        self.a, self.b = normal(L, r, K, size=K ** -0.5), normal(L, N, r, size=r ** -0.5)
        self.scale = (0.5 + torch.rand(L, generator=g)).cuda()
        self.number = torch.randint(-1, L, (T, 1), generator=g).int().cuda()
        self.offsets = torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32).cuda()
        self.grad_out, self.grad_weights = normal(T, N), normal(T, k)
        self.grad_loss = normal(len(lengths), size=30.0)

    def run(self):
        """(out, weights, experts, loss, counts), (grad_x, grad_a, grad_b, grad_router)."""
        layout = binding.experts_layout(self.number, self.L)
        y = binding.linear(self.x, self.w)
        out = binding.adapters_linear(self.x, self.a, self.b, layout, y, scale=self.scale, out=y)
        logits = binding.linear(out, self.router)
        weights, experts = binding.route_experts(logits, self.k, score=self.score)
        loss, counts = binding.balance_loss(logits, experts, score=self.score, offsets=self.offsets)
        grad_logits = binding.balance_loss_backward(self.grad_loss, logits, experts, counts, score=self.score,
                                                    offsets=self.offsets, grad_weights=self.grad_weights)
        grad_out = self.grad_out + binding.linear(grad_logits, self.router.t().contiguous())
        grad_router = binding.linear(grad_logits.t().contiguous(), out.t().contiguous())
        shared = binding.linear(grad_out, self.w.t().contiguous())
        grads = binding.adapters_linear_backward(grad_out, self.x, self.a, self.b, layout, shared, scale=self.scale)
        return (out, weights, experts, loss, counts), (*grads, grad_router)

    def plain(self, experts):
        """The same in 64 bits with autograd, for this choice of experts."""
        x, a, b, w, router = (t.double().cpu().requires_grad_() for t in (self.x, self.a, self.b, self.w, self.router))
        number, experts = self.number[:, 0].cpu(), experts.cpu().long()
        out = x @ w.t()
        for l in range(self.L):
            mine = (number == l).double()[:, None]
            out = out + mine * float(self.scale[l]) * (x @ a[l].t()) @ b[l].t()
        logits = out @ router.t()
        s = torch.softmax(logits, -1) if self.score == "softmax" else torch.sigmoid(logits)
        chosen = s.gather(1, experts)
        weights = chosen / chosen.sum(-1, keepdim=True)
        p = s / s.sum(-1, keepdim=True)
        ends, E, losses, counts = self.offsets.tolist(), router.shape[0], [], []
        for lo, hi in zip(ends, ends[1:]):
            c = torch.bincount(experts[lo:hi].flatten(), minlength=E)
            counts.append(c)
            losses.append(E / (self.k * max(hi - lo, 1) ** 2) * (c * p[lo:hi].sum(0)).sum())
        loss, counts = torch.stack(losses), torch.stack(counts)
        total = ((out * self.grad_out.double().cpu()).sum() + (weights * self.grad_weights.double().cpu()).sum()
                 + (loss * self.grad_loss.double().cpu()).sum())
        total.backward()
        return (out, weights, loss, counts), (x.grad, a.grad, b.grad, router.grad)


def close(got, want, bound=1e-3):
    want = want.detach()
    off, size = (got.double().cpu() - want).norm().item(), want.norm().item()
    assert off <= bound * size, (off, size)


STEPS = [(1, 2, 8, 256, 256, 8, 2, [1]), (70, 5, 8, 256, 256, 16, 2, [30, 0, 37]),
         (900, 4, 16, 256, 264, 64, 6, [500, 1, 300]), (1700, 3, 32, 200, 256, 33, 4, [900, 800])]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,L,r,K,N,E,k,lengths", STEPS)
def test_training_step(T, L, r, K, N, E, k, lengths, score):
    step = Step(T, L, r, K, N, E, k, lengths, score)
    (out, weights, experts, loss, counts), grads = step.run()
    (out64, weights64, loss64, counts64), grads64 = step.plain(experts)
    close(out, out64)
    close(weights, weights64)
    close(loss, loss64)
    assert torch.equal(counts.cpu().long(), counts64)
    for got, want in zip(grads, grads64):
        close(got, want)
    assert binding.check_device_error(None) == binding.IMC_OK


def test_training_step_captured():
    """The whole step in a graph, replayed on other tokens, adapters and sequences."""
    step = Step(900, 4, 16, 256, 264, 64, 6, [500, 1, 300], "softmax")
    step.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        values, grads = step.run()
    other = Step(900, 4, 16, 256, 264, 64, 6, [10, 700, 190], "softmax", seed=1)
    for name in ("x", "number", "offsets", "grad_out"):
        getattr(step, name).copy_(getattr(other, name))
    graph.replay()
    eager_values, eager_grads = step.run()
    torch.cuda.synchronize()
    for got, want in zip((*values, *grads), (*eager_values, *eager_grads)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T", [1, 24, 700])
def test_serving_step(T, dtype):
    """A 4-bit projection and the requests' adapters in place on its result, captured once."""
    c = Case(T, T, 6, 16, 256, 384, dtype)
    w = binding.quantize_mxfp4(torch.randn(384, 256, generator=torch.Generator().manual_seed(1)).cuda())
    number = c.which[:, None].clone()

    def step():
        layout = binding.experts_layout(number, 6)
        y = binding.linear_mxfp4(c.x, w, out_dtype=dtype)
        return binding.adapters_linear(c.x, c.a, c.b, layout, y, scale=c.scale, out=y)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2):
        other = Case(seed + 7, T, 6, 16, 256, 384, dtype)
        c.x.copy_(other.x)
        c.which = other.which
        number.copy_(other.which[:, None])
        graph.replay()
        c.base = binding.linear_mxfp4(c.x, w, out_dtype=dtype)
        within(out, *c.forward64(), dtype)
