"""Gradients of routing weights whose chosen experts have scores below fp32's smallest normal
number beside others of ordinary size (chosen by a bias, say): w_i = s_i / sum of the chosen s
is an ordinary number, and so is its gradient, w_e (g_e - sum g w) for the chosen experts.

Scores are 16 * 2^-23 of their value off as elsewhere, and 2^-149 by fp32's smallest step: with
q the smallest chosen score 2^-149 / q relative, which enters an output through s_e, the sum and
the inner sum (four times at most, k terms each having no more than its share).
"""
import numpy as np
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding
from test_gpu_adapters import f64
from test_gpu_balance import EPS, TYPES, Case
from test_gpu_experts import scores64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("at", [-60.0, -86.0, -90.0])
def test_chosen_scores_near_zero(at, score, dtype):
    T, E, k = 30, 48, 3
    c = Case(T, T, E, k, score, dtype, skew=0.0)
    rows = [2, 9, 29]
    g = torch.Generator().manual_seed(5)
    for t in rows:
        at_these = torch.randperm(E, generator=g)[:k]
        c.logits[t] = 0.0
        c.logits[t, at_these] = (at + torch.randint(-2, 3, (k,), generator=g)).to(dtype).cuda()
        c.experts[t] = at_these.int().cuda()
    c.grad_loss.zero_()
    _, counts = c.forward()
    both = c.backward(counts, True)
    within(both, c, scores64(f64(c.logits), score))
    routed = binding.route_experts_backward(c.grad_weights, c.logits, c.experts, score=score)
    s = scores64(f64(c.logits), score)
    if score == "sigmoid":  # moe_route's are 1 / (1 + e^-x), 0 where e^-x passes fp32's range
        s = np.where(f64(c.logits) < -np.log(2.0 ** 128), 0.0, s)
    within(routed, c, s)


def within(got, c, s):
    e, gw, soft = c.experts.cpu().numpy(), c.grad_weights.double().cpu().numpy(), c.score == "softmax"
    picked = np.take_along_axis(s, e, 1)
    total = picked.sum(-1, keepdims=True)
    w = picked / np.where(total == 0, 1, total)
    inner = (gw * w).sum(-1, keepdims=True)
    want, size = np.zeros_like(s), np.zeros_like(s)
    np.put_along_axis(want, e, w * (gw - inner) * (1.0 if soft else 1 - picked), 1)
    # (softmax: the kernels' inner sum over the chosen, 0 in exact numbers, is off by a few roundings of
    # its terms, and reaches every expert by its score)
    terms = w * (np.abs(gw) + (np.abs(gw) * w).sum(-1, keepdims=True))
    np.put_along_axis(size, e, terms, 1)
    if soft:
        size = size + s * terms.sum(-1, keepdims=True)
    lost = 4 * 2.0 ** -149 / np.where(picked > 0, picked, 1).min(-1, keepdims=True)
    tol = ((48 + c.E / 32) * EPS + lost) * size
    tol = tol + torch.finfo(c.dtype).eps / 2 * (np.abs(want) + tol) + (2.0 ** -24 if c.dtype == torch.float16 else 1e-37)
    off = np.abs(f64(got) - want)
    assert (off <= tol).all(), (off - tol).max()
