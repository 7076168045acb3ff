"""Logits of tokens in no sequence (padding) may hold anything: the loss, the counts and the
other tokens' gradients do not see them, and their own gradient of the loss is 0."""
import pytest
import torch

from test_gpu_balance import TYPES, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("lengths,tail", [([3, 20, 0, 9], 5), ([40, 700, 100], 60)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), "lowest"])
def test_padding_of_any_value(value, lengths, tail, score, dtype):
    T = sum(lengths) + tail
    c = Case(T, T, 40, 3, score, dtype, lengths)
    loss, counts = c.forward()
    good = c.backward(counts, False)
    inside = slice(lengths[0], T - tail)
    if value == "lowest":
        value = torch.finfo(dtype).min
    c.logits[:lengths[0]] = value
    c.logits[T - tail:, ::2] = value
    again, counts_again = c.forward()
    assert torch.equal(again, loss) and torch.equal(counts_again, counts)
    got = c.backward(counts, False)
    assert torch.equal(got[inside], good[inside])
    assert not got[:lengths[0]].any() and not got[T - tail:].any()


def test_no_sequence_at_all():
    c = Case(1, 30, 24, 2, "softmax", torch.float32, [9])
    c.logits[4, 5] = float("nan")
    loss, counts = c.forward()
    assert not c.backward(counts, False).any()


def test_routing_weights_of_padding():
    """With the routing weights' gradient the padding has that one alone."""
    from addmm_implicit_im2col_gb300 import binding
    c = Case(2, 60, 24, 3, "sigmoid", torch.float32, [4, 30, 10])
    c.grad_weights[50:] = 0  # no loss reads these tokens
    _, counts = c.forward()
    got = c.backward(counts, True)
    routed = binding.route_experts_backward(c.grad_weights, c.logits, c.experts, score="sigmoid")
    assert not got[50:].any() and torch.allclose(got[:4], routed[:4], rtol=1e-4, atol=1e-7)
