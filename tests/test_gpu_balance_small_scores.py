"""The balance loss and its gradient for tokens whose sigmoids all lie near or below fp32's
smallest numbers (sums below 2^-128 have no reciprocal in fp32): their quotients are ordinary
numbers all the same.  Tolerances are those of the other balance tests (test_gpu_balance.py):
sigmoids of logits below -70 are e^x to 2^-100, and the quotients the softmax.
"""
import numpy as np
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding
from test_gpu_adapters import f64
from test_gpu_balance import EPS, TYPES, Case

pytestmark = pytest.mark.gpu


def far(seed, T, E, k, dtype, rows, at, lengths=None):
    """Ordinary logits, but for these rows, whose logits lie around `at`."""
    c = Case(seed, T, E, k, "sigmoid", dtype, lengths)
    g = torch.Generator().manual_seed(seed + 100)
    c.logits[rows] = (at + 1.5 * torch.randn(len(rows), E, generator=g)).to(dtype).cuda()
    c.experts = c.logits.float().topk(k, -1).indices.int().contiguous()
    return c


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("at", [-66.0, -72.0, -84.0, -90.0, -95.0, -99.0])
@pytest.mark.parametrize("T,E,k", [(40, 16, 2), (40, 64, 4), (33, 300, 6), (900, 64, 4), (700, 1024, 8)])
def test_tokens_far_from_zero(T, E, k, at, dtype):
    far(T + E, T, E, k, dtype, [0, 7, T - 1], at).check()


def test_every_token_of_a_sequence():
    far(1, 60, 32, 3, torch.float32, list(range(20, 50)), -95.0, [0, 20, 30]).check()
    far(2, 900, 32, 3, torch.float32, list(range(300, 700)), -95.0, [0, 300, 400]).check()


@pytest.mark.parametrize("T", [40, 900])
def test_sigmoids_that_are_zero_in_fp32(T):
    """The loss and its gradient follow the definition there too; the routing weights are 0 (route_experts'
    are), and so is their gradient."""
    c = far(3, T, 48, 4, torch.float32, [5, 11], -130.0)
    loss, counts = c.forward()
    want = c.loss64()[0]
    assert (np.abs(f64(loss) - want) <= (49 + (c.E / 32 + 8) / 2) * EPS * want).all()
    alone = c.backward(counts, False)
    v, tol = c.grad64(False)
    assert (np.abs(f64(alone) - v) <= tol).all()
    both = c.backward(counts, True)
    assert torch.equal(both[[5, 11]], alone[[5, 11]])
    assert not binding.route_experts(c.logits, 4, score="sigmoid")[0][[5, 11]].any()
