"""The routers' balance loss, counts and gradient against the definition in 64 bits.

Tolerances.  A score is off by at most 16 * 2^-23 of its value (as in the routing tests; the
sigmoid's division by the sum adds E / 32 + 8 roundings of 2^-24), a lane's fp32 sums of up to
64 scores by 64 * 2^-24, sums beyond are in 64 bits and the loss is rounded once: loss within
(16 + (E / 32 + 8) / 2 + 32 + 1) * 2^-23 of itself, since its terms have one sign.
Gradient: u is two roundings and a division off, the inner sum E / 32 + 8 roundings; every term
is one of the sums of magnitudes below, of which c = (48 + E / 32) * 2^-23 is allowed, then one
rounding to the logits' type.
"""
import random

import numpy as np
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding
from test_gpu_adapters import TINY, f64
from test_gpu_experts import scores64

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -23
TYPES = [torch.float32, torch.bfloat16, torch.float16]


class Case:
    def __init__(self, seed, T, E, k, score, dtype=torch.float32, lengths=None, skew=0.5):
        g = torch.Generator().manual_seed(seed)
        self.T, self.E, self.k, self.score, self.dtype = T, E, k, score, dtype
        x = 1.5 * torch.randn(T, E, generator=g) + skew * torch.randn(E, generator=g)
        self.logits = x.to(dtype).cuda()
        self.experts = self.logits.float().topk(k, -1).indices.int().contiguous()
        self.offsets = None
        if lengths is not None:
            self.offsets = torch.tensor(np.concatenate([[lengths[0]], lengths[0] + np.cumsum(lengths[1:])]),
                                        dtype=torch.int32).cuda()
        self.S = 1 if lengths is None else len(lengths) - 1
        self.grad_loss = (100 * torch.randn(self.S, generator=g)).cuda()
        self.grad_weights = torch.randn(T, k, generator=g).cuda()

    def spans(self):
        if self.offsets is None:
            return [(0, self.T)]
        o = np.clip(self.offsets.cpu().numpy(), 0, self.T)
        return [(o[i], max(o[i], o[i + 1])) for i in range(self.S)]

    def loss64(self):
        s = scores64(f64(self.logits), self.score)
        total = s.sum(-1, keepdims=True)
        p = s / np.where(total == 0, 1, total)
        experts = self.experts.cpu().numpy()
        loss, counts = np.zeros(self.S), np.zeros((self.S, self.E), dtype=np.int64)
        for i, (lo, hi) in enumerate(self.spans()):
            e = experts[lo:hi].ravel()
            counts[i] = np.bincount(e[(e >= 0) & (e < self.E)], minlength=self.E)
            if hi > lo:
                loss[i] = self.E / (self.k * float(hi - lo) ** 2) * (counts[i] * p[lo:hi].sum(0)).sum()
        return loss, counts, s, p, np.where(total == 0, 1, total)

    def grad64(self, weights, renormalize=True, scale=1.0):
        loss, counts, s, p, total = self.loss64()
        u, coef = np.zeros((self.T, self.E)), self.grad_loss.double().cpu().numpy()
        for i, (lo, hi) in enumerate(self.spans()):
            if hi > lo:
                u[lo:hi] = coef[i] * self.E / (self.k * float(hi - lo) ** 2) * counts[i]
        inner = (u * p).sum(-1, keepdims=True)
        soft = self.score == "softmax"
        rest = s if soft else s * (1 - s)
        out = (u - inner) * rest if soft else (u - inner) / total * rest
        size = (np.abs(u) + (np.abs(u) * p).sum(-1, keepdims=True)) * rest / (1 if soft else total)
        if weights:
            g, e = self.grad_weights.double().cpu().numpy(), self.experts.cpu().numpy()
            ok = (e >= 0) & (e < self.E)
            picked = np.where(ok, np.take_along_axis(s, np.where(ok, e, 0), 1), 0.0)
            S = picked.sum(-1, keepdims=True)
            S = np.where(S == 0, 1, S)
            if renormalize:
                d = (g - (g * picked).sum(-1, keepdims=True) / S) / S
                dsize = (np.abs(g) + (np.abs(g) * picked).sum(-1, keepdims=True) / S) / S
            else:
                d, dsize = g, np.abs(g)
            d, dsize = np.where(ok, d, 0) * scale, np.where(ok, dsize, 0) * abs(scale)
            full, fsize = np.zeros_like(s), np.zeros_like(s)
            for t in range(self.T):
                np.add.at(full[t], e[t][ok[t]], d[t][ok[t]])
                np.add.at(fsize[t], e[t][ok[t]], dsize[t][ok[t]])
            if soft:
                fsize = fsize + (dsize * picked).sum(-1, keepdims=True)
                full = full - (d * picked).sum(-1, keepdims=True)
            out, size = out + full * rest, size + fsize * rest
        tol = (48 + self.E / 32) * EPS * size
        return out, tol + torch.finfo(self.dtype).eps / 2 * (np.abs(out) + tol) + TINY[self.dtype]

    def forward(self):
        return binding.balance_loss(self.logits, self.experts, score=self.score, offsets=self.offsets)

    def backward(self, counts, weights, **kw):
        return binding.balance_loss_backward(self.grad_loss, self.logits, self.experts, counts, score=self.score,
                                             offsets=self.offsets,
                                             grad_weights=self.grad_weights if weights else None, **kw)

    def check(self):
        loss, counts = self.forward()
        want, want_counts = self.loss64()[:2]
        assert loss.dtype == torch.float32 and counts.dtype == torch.int32
        assert np.array_equal(counts.cpu().numpy(), want_counts)
        assert (np.abs(f64(loss) - want) <= (49 + (self.E / 32 + 8) / 2) * EPS * want).all()
        for weights, renormalize, scale in ((False, True, 1.0), (True, True, 1.0), (True, False, 2.5)):
            got = self.backward(counts, weights, renormalize=renormalize, scale=scale)
            v, tol = self.grad64(weights, renormalize, scale)
            assert got.dtype == self.dtype
            off = np.abs(f64(got) - v)
            worst = np.unravel_index(np.argmax(off - tol), off.shape)
            assert (off <= tol).all(), f"{worst}: off by {off[worst]}, allowed {tol[worst]}"


SIZES = [(1, 1, 1), (1, 8, 2), (5, 4, 4), (64, 64, 4), (65, 33, 5), (300, 100, 8), (1000, 128, 8), (513, 256, 8),
         (40, 300, 6), (33, 520, 32), (70, 1024, 8), (5000, 16, 2)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_one_sequence(T, E, k, score, dtype):
    Case(T + E, T, E, k, score, dtype).check()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("lengths,tail", [([0, 5, 0, 9, 1], 0), ([3, 100, 0, 0, 1, 200], 17), ([0] + [1] * 70, 3),
                                          ([0, 0], 6), ([7], 2), ([0] + [3, 0, 40] * 30, 0), ([0, 2000, 3, 500], 9)])
def test_sequences(lengths, tail, score):
    """Sequences of any length, empty ones, rows before the first and behind the last."""
    T = sum(lengths) + tail
    Case(T, T, 48, 4, score, torch.bfloat16, lengths).check()


@pytest.mark.parametrize("seed", range(16))
def test_any_sizes(seed):
    r = random.Random(seed)
    E = r.randint(1, 1024 if seed % 4 == 0 else 260)
    T = int(np.exp(r.uniform(0, 7.5)))
    lengths = None
    if seed % 2:
        cuts = sorted(r.randint(0, T) for _ in range(r.randint(0, 40)))
        lengths = [0] + list(np.diff([0] + cuts)) if cuts else None
    Case(seed, T, E, r.randint(1, min(32, E)), r.choice(["softmax", "sigmoid"]), TYPES[seed % 3], lengths).check()


def test_long():
    """A long sequence (sums of many scores), alone and cut into a few."""
    Case(1, 40000, 64, 4, "sigmoid").check()
    Case(2, 40000, 40, 2, "softmax", torch.float32, [0, 30000, 1, 9000]).check()


@pytest.mark.parametrize("lengths", [[0] + [17] * 150, [5, 0, 0, 1500, 0, 1, 1, 1, 900, 0, 64, 0], [2900, 10, 20],
                                     [0] + [1] * 900 + [2000], [0] + [0] * 400 + [2500] + [0] * 300])
def test_many_tokens_in_sequences(lengths):
    """The form for many tokens, whose blocks each meet several sequences, or none."""
    T = sum(lengths) + 40
    Case(T, T, 24, 3, "sigmoid", torch.float32, lengths).check()


def test_offsets_outside_the_tokens():
    c = Case(3, 50, 16, 2, "softmax", torch.float32, [0, 20, 30])
    want = c.forward()
    c.offsets = torch.tensor([-7, 20, 999], dtype=torch.int32, device="cuda")
    assert all(torch.equal(p, q) for p, q in zip(c.forward(), want))
    c.check()


def test_slots_of_no_expert():
    c = Case(4, 90, 12, 3, "sigmoid")
    c.experts[::3, 1] = -1
    c.experts[5] = 12
    c.check()


def test_even_routing_has_loss_one():
    E, k = 32, 4
    experts = (torch.arange(64 * k, device="cuda") % E).view(64, k).int()
    loss, counts = binding.balance_loss(torch.zeros(64, E, device="cuda"), experts)
    assert abs(float(loss) - 1) <= 1e-5 and bool((counts == 8).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_rows_without_scores(score):
    """Logits of -inf alone have scores of 0 and no gradient; some of them are like others."""
    c = Case(5, 40, 16, 2, score)
    c.logits[7] = float("-inf")
    c.logits[9, 3:] = float("-inf")
    c.check()
    loss, counts = c.forward()
    assert not c.backward(counts, True)[7].any()


def test_nan_stays_in_its_sequence_and_row():
    c = Case(6, 60, 16, 2, "softmax", torch.float32, [0, 20, 40])
    loss, counts = c.forward()
    good = c.backward(counts, True)
    c.logits[25, 3] = float("nan")
    bad, _ = c.forward()
    assert torch.isnan(bad[1]) and torch.equal(bad[0], loss[0])
    got, keep = c.backward(counts, True), torch.arange(60, device="cuda") != 25
    assert torch.equal(got[keep], good[keep]) and torch.isnan(got[25]).all()


def test_strided_logits():
    c = Case(7, 70, 24, 3, "softmax", torch.bfloat16)
    wide = torch.full((70, 31), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 5:29] = c.logits
    c.logits = wide[:, 5:29]
    c.check()


def test_sum_of_both_gradients():
    """With grad_weights the result is the sum of the two gradients."""
    c = Case(8, 200, 64, 6, "sigmoid")
    _, counts = c.forward()
    both = c.backward(counts, True, scale=1.5)
    apart = c.backward(counts, False) + binding.route_experts_backward(c.grad_weights, c.logits, c.experts,
                                                                       score="sigmoid", scale=1.5)
    assert torch.allclose(both, apart, rtol=1e-4, atol=1e-6)


def test_gradient_against_differences():
    c = Case(9, 12, 6, 2, "softmax", torch.float32, [0, 5, 7])
    _, counts = c.forward()
    grad = f64(c.backward(counts, False))
    g = c.grad_loss.double().cpu().numpy()
    kept = c.logits.clone()
    for t, e in ((0, 0), (4, 3), (5, 1), (11, 5)):
        ends = []
        for step in (2.0 ** -5, -2.0 ** -5):
            c.logits.copy_(kept)
            c.logits[t, e] += step
            ends.append((f64(c.forward()[0]) * g).sum())
        # third derivatives of a softmax (below 1) of a loss of some units times 100, step^2 / 6;
        # the loss's own error 1e-5 of 100s over the step
        assert abs((ends[0] - ends[1]) / 2.0 ** -4 - grad[t, e]) <= 100 * 6 * 2.0 ** -10 / 6 + 0.2


def test_twice_the_same_bits_on_any_stream_and_replayed():
    c = Case(10, 3000, 128, 8, "sigmoid", torch.float32, [0, 1000, 1500])

    def both():
        loss, counts = c.forward()
        return [loss, counts, c.backward(counts, True)]

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    c.logits.copy_(Case(11, 3000, 128, 8, "sigmoid").logits)
    eager = both()
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(outs, eager))


def test_empty_calls():
    x, e = torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    loss, counts = binding.balance_loss(x, e)
    assert loss.tolist() == [0.0] and not counts.any() and counts.shape == (1, 8)
    assert binding.balance_loss_backward(loss, x, e, counts).shape == (0, 8)
    c = Case(12, 5, 8, 2, "softmax", torch.float32, [3])  # no sequence at all
    loss, counts = c.forward()
    assert loss.shape == (0,) and counts.shape == (0, 8)
    assert not c.backward(counts, False).any()


def test_refused_by_the_torch_level():
    c = Case(1, 6, 8, 2, "softmax", torch.float32, [0, 3, 3])
    with pytest.raises(KeyError):
        binding.balance_loss(c.logits, c.experts, score="other")
    with pytest.raises(ValueError):
        binding.balance_loss(c.logits, c.experts.long())
    with pytest.raises(ValueError):
        binding.balance_loss(c.logits, c.experts[:5].contiguous())
    with pytest.raises(ValueError):
        binding.balance_loss(c.logits, c.experts, offsets=c.offsets.long())
    with pytest.raises(ValueError):
        binding.balance_loss(c.logits, c.experts, offsets=c.offsets[None])
    with pytest.raises(ValueError):
        binding.balance_loss(c.logits, c.experts, offsets=c.offsets.cpu())
    _, counts = c.forward()
    with pytest.raises(ValueError):
        binding.balance_loss_backward(c.grad_loss[:1], c.logits, c.experts, counts, offsets=c.offsets)
    with pytest.raises(ValueError):
        binding.balance_loss_backward(c.grad_loss, c.logits, c.experts, counts[:1], offsets=c.offsets)
    with pytest.raises(ValueError):
        binding.balance_loss_backward(c.grad_loss, c.logits, c.experts, counts, offsets=c.offsets,
                                      grad_weights=c.grad_weights.half())


@pytest.mark.parametrize("T", [639, 640, 641, 642])
def test_around_the_rule_for_many_tokens(T):
    """One launch up to 640 tokens, chunks and a join beyond."""
    assert (binding.moe_balance_workspace_bytes(T, 1, 40) > 0) == (T > 640)
    Case(T, T, 40, 3, "softmax").check()


@pytest.mark.parametrize("S,T", [(15, 960), (15, 961), (40, 2561), (1025, 2050), (400, 401)])
def test_around_the_rule_for_many_sequences(S, T):
    """Chunks where a sequence has more than 64 tokens on average; one of them has most here."""
    assert (binding.moe_balance_workspace_bytes(T, S, 24) > 0) == (T in (961, 2561))
    Case(S, T, 24, 2, "sigmoid", lengths=[0] + [1] * (S - 1) + [T - S + 1]).check()
