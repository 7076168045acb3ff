"""The balance loss where its scores and its last factor are exact, so that the sums alone decide.

A token with 2^j equal logits and -inf elsewhere has the scores 2^-j and 0, exactly; with 2^i
experts and 2^m tokens E / (k n^2) is a power of two.  The sums P of an expert's scores are exact
in a pair of fp32 numbers.  What is left is the sum of c * P over the experts, kept as a pair to
2^-46 of itself for each of a few terms (24 bits and the rounding errors, exactly), and one
rounding: the loss is within half a step of its value, 2^-24, and 2^-40 more is allowed.
"""
import numpy as np
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding

pytestmark = pytest.mark.gpu


def check(seed, n, S, E, used):
    """S sequences of n tokens, whose slots are the experts `used` or none."""
    g = torch.Generator().manual_seed(seed)
    T = n * S
    live = 2 ** torch.randint(0, E.bit_length(), (T,), generator=g)
    place = torch.rand(T, E, generator=g).argsort(1)
    place[torch.arange(T), place.argmin(1)] = place[:, used[0]]
    place[:, used[0]] = 0  # the first of them has a score in every token
    logits = torch.where(place < live[:, None], 0.0, float("-inf"))
    share = torch.rand(S, generator=g).repeat_interleave(n)
    number = torch.tensor(used)[torch.randint(0, len(used), (T,), generator=g)]
    experts = torch.where(torch.rand(T, generator=g) < share, number, -1).int()
    offsets = torch.arange(S + 1, dtype=torch.int32) * n
    loss, counts = binding.balance_loss(logits.cuda(), experts[:, None].contiguous().cuda(), offsets=offsets.cuda())
    score = np.where(np.isfinite(logits.numpy()), 1.0 / live.double().numpy()[:, None], 0.0).reshape(S, n, E).sum(1)
    c = np.stack([(experts.numpy().reshape(S, n) == e).sum(1) for e in range(E)], 1)
    assert np.array_equal(counts.cpu().numpy(), c)
    want = E / n ** 2 * (c * score).sum(1)  # exact in 64 bits
    off = np.abs(loss.double().cpu().numpy() - want)
    assert (off <= (2.0 ** -24 + 2.0 ** -40) * want).all(), (off / np.maximum(want, 1e-300)).max() * 2 ** 24


@pytest.mark.parametrize("n,S", [(64, 9), (512, 40), (2048, 1), (4096, 16)])
@pytest.mark.parametrize("E,used", [(32, [5]), (256, [5]), (256, [5, 6, 133, 255])])
def test_loss_is_rounded_once(n, S, E, used):
    check(n + S + E, n, S, E, used)


@pytest.mark.parametrize("E,used", [(64, [3]), (512, [5, 261]), (1024, [5, 261, 517, 773]), (1024, [1, 2, 258, 1023])])
def test_loss_of_few_tokens_is_rounded_once(E, used):
    """One launch; a thread has the experts e, e + 256, ..."""
    for seed in range(24):
        check(seed, 512, 1, E, used)
