"""Expert routing, layout, products and weighted sum against 64-bit references.

Tolerances.  Scores are a few fp32 operations (exp within 2 units in the last
place, a sum of E terms in a tree, one or two divisions): 16 * 2^-23 relative
covers them, with the choice's sum of k scores.  Products as in the MXFP4
tests.  Weighted sums: k (forward) or N / 32 + 8 (backward, a warp's tree)
roundings of 2^-24 of the sum of magnitudes, one rounding to the output's type.
"""
import random

import numpy as np
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding
from test_gpu_mxfp4 import HALF_ULP, check, f64, mx_blocks, product_case, spread

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -23


def scores64(x, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-x))
    m = x.max(-1, keepdims=True)
    e = np.exp(np.where(np.isneginf(m), -np.inf, x - np.where(np.isneginf(m), 0, m)))
    s = e.sum(-1, keepdims=True)
    return e / np.where(s == 0, 1, s)


def route64(x, k, bias, score, groups, top_groups, renormalize, scale):
    s = scores64(x, score)
    c = s if bias is None else s + bias
    T, E = x.shape
    experts = np.zeros((T, k), dtype=np.int64)
    for t in range(T):
        key = c[t].copy()
        if groups > 1:
            per = key.reshape(groups, -1)
            two = np.sort(per, -1)[:, -2:].sum(-1)
            kept = np.argsort(-two, kind="stable")[:top_groups]
            out = np.ones(groups, dtype=bool)
            out[kept] = False
            key[np.repeat(out, E // groups)] = -np.inf
        experts[t] = np.argsort(-key, kind="stable")[:k]
    w = np.take_along_axis(s, experts, 1)
    if renormalize:
        total = w.sum(-1, keepdims=True)
        w = np.where(total == 0, 0, w / np.where(total == 0, 1, total))
    return w * scale, experts


def near(s):
    """Rows with two values closer than 1e-6 that are not equal (equal ones are exact ties)."""
    d = np.diff(np.sort(s, -1), axis=-1)
    return ((d < 1e-6) & (d > 0)).any(-1)


def clear_logits(seed, T, E, bias, k, score, groups, top_groups, dtype=torch.float32):
    """Logits whose choice no rounding can turn (rows that one could are drawn again)."""
    g = torch.Generator().manual_seed(seed)
    x = (1.5 * torch.randn(T, E, generator=g)).to(dtype)
    for _ in range(50):
        s = scores64(f64(x), score) + (0 if bias is None else bias)
        bad = np.zeros(T, dtype=bool)
        if groups > 1:
            bad |= near(np.sort(s.reshape(T, groups, -1), -1)[..., -2:].sum(-1))
        bad |= near(s if E <= 64 or groups > 1 else np.sort(s, -1)[:, -(k + 1):])
        if not bad.any():
            return x.cuda()
        at = torch.from_numpy(bad)
        x[at] = (1.5 * torch.randn(int(bad.sum()), E, generator=g)).to(dtype)
    raise AssertionError("no clear logits")


ROUTES = [(1, 1, 1, "softmax", False, 1, 1), (5, 8, 2, "softmax", False, 1, 1),
          (33, 8, 8, "sigmoid", True, 1, 1), (64, 33, 5, "softmax", True, 1, 1),
          (257, 64, 6, "sigmoid", True, 8, 3), (100, 48, 4, "softmax", False, 4, 2),
          (50, 128, 8, "sigmoid", True, 4, 2), (77, 100, 7, "sigmoid", False, 5, 5),
          (40, 256, 8, "sigmoid", True, 8, 4), (3, 32, 4, "softmax", True, 32, 8),
          (19, 24, 3, "softmax", False, 24, 4), (8, 132, 3, "softmax", True, 4, 2),
          (30, 255, 6, "sigmoid", True, 5, 1), (12, 300, 4, "sigmoid", True, 10, 2),
          (9, 1024, 8, "sigmoid", True, 32, 3)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k,score,use_bias,groups,top_groups", ROUTES)
def test_route(T, E, k, score, use_bias, groups, top_groups, renormalize, dtype):
    bias = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E)) if use_bias else None
    b64 = None if bias is None else f64(bias)
    if E == 1 or (groups == E and not use_bias):
        x = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).cuda()
    else:
        x = clear_logits(T + E, T, E, b64, k, score, groups, top_groups, dtype)
    w, experts = binding.route_experts(x, k, None if bias is None else bias.cuda(), score=score,
                                       groups=groups, top_groups=top_groups,
                                       renormalize=renormalize, scale=2.5)
    w64, e64 = route64(f64(x), k, b64, score, groups, top_groups, renormalize, 2.5)
    assert np.array_equal(experts.cpu().numpy(), e64)
    assert np.abs(f64(w) - w64).max() <= 16 * EPS * 2.5
    assert (np.abs(f64(w) - w64) <= 16 * EPS * np.abs(w64) + 1e-30).all()


@pytest.mark.parametrize("seed", range(24))
def test_route_of_any_sizes(seed):
    """Sizes, groups and forms drawn over their whole range."""
    r = random.Random(seed)
    groups = r.choice([1, 2, 3, 4, 5, 7, 8, 16, 32])
    E = groups * r.randint(1, (512 if seed % 3 else 1024) // groups)
    top_groups = r.randint(1, groups)
    k = r.randint(1, min(32, E // groups * top_groups))
    score = r.choice(["softmax", "sigmoid"])
    bias = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(seed))
    T = r.randint(1, 40)
    x = clear_logits(seed, T, E, f64(bias), k, score, groups, top_groups, torch.float32)
    w, experts = binding.route_experts(x, k, bias.cuda(), score=score, groups=groups, top_groups=top_groups)
    w64, e64 = route64(f64(x), k, f64(bias), score, groups, top_groups, True, 1.0)
    assert np.array_equal(experts.cpu().numpy(), e64)
    assert (np.abs(f64(w) - w64) <= 16 * EPS * np.abs(w64) + 1e-30).all()


@pytest.mark.parametrize("seed", range(24))
def test_experts_linear_of_any_sizes(seed):
    r = random.Random(100 + seed)
    E, T = r.randint(1, 40), int(2 ** r.uniform(0, 9.5))
    k, N, K = r.randint(1, min(8, E)), int(2 ** r.uniform(0, 9)), int(2 ** r.uniform(0, 11))
    per_slot, dtype = r.random() < 0.5, r.choice([torch.float32, torch.bfloat16])
    experts = some_experts(seed, T, k, E, r.random() < 0.5)
    x, w = spread(1, T * k if per_slot else T, K, dtype), spread(2, E * N, K).view(E, N, K)
    got = binding.experts_linear_mxfp4(x, binding.quantize_mxfp4(w), binding.experts_layout(experts, E))
    xq, flat = mx_blocks(f64(x))[0], experts.reshape(-1).cpu().numpy()
    y, s = np.zeros((T * k, N)), np.zeros((T * k, N))
    for e in range(E):
        at = np.nonzero(flat == e)[0]
        if len(at):
            y[at], s[at] = product_case(xq[at if per_slot else at // k], mx_blocks(f64(w[e]))[0])
    check(got, y, s, K, dtype)
    assert binding.check_device_error() == binding.IMC_OK


@pytest.mark.parametrize("E", [300, 512, 1024])
def test_route_many_experts(E):
    x = clear_logits(E, 20, E, None, 32, "softmax", 1, 1)
    w, experts = binding.route_experts(x, 32)
    w64, e64 = route64(f64(x), 32, None, "softmax", 1, 1, True, 1.0)
    assert np.array_equal(experts.cpu().numpy(), e64)
    assert (np.abs(f64(w) - w64) <= 16 * EPS * w64).all()


def test_route_ties_and_special_rows():
    E, inf, nan = 40, float("inf"), float("nan")
    x = torch.zeros(8, E)
    x[1, 3:] = 1.0                # equal logits: the lowest indices
    x[2] = -inf                   # a row without a score
    x[3], x[3, 7] = -inf, 0.5     # one expert alone
    x[4, 11] = nan
    x[5], x[5, [4, 9]] = -1e30, 2.0
    x[6] = torch.arange(E).float().neg()
    x[7, :] = torch.tensor([1.0, -1.0]).repeat(E // 2)
    w, e = binding.route_experts(x.cuda(), 4)
    e, w = e.cpu().tolist(), w.cpu()
    assert e[0] == [0, 1, 2, 3] and e[1] == [3, 4, 5, 6] and e[2] == [0, 1, 2, 3]
    assert e[3][0] == 7 and e[3][1:] == [0, 1, 2] and e[5][:2] == [4, 9] and e[6] == [0, 1, 2, 3]
    assert e[7] == [0, 2, 4, 6]
    assert w[0].tolist() == [0.25] * 4 and w[2].tolist() == [0.0] * 4
    assert w[3].tolist() == [1.0, 0, 0, 0]
    assert w[4].isnan().all() and e[4] == [0, 1, 2, 3]  # softmax of a NaN: every score is NaN
    assert w[5, :2].tolist() == [0.5, 0.5]
    # sigmoid scores are apart: a NaN is chosen last
    w, e = binding.route_experts(x[4:5, :32].cuda(), 32, score="sigmoid", renormalize=False)
    assert sorted(e[0].tolist()) == list(range(32)) and e[0, -1].item() == 11 and w[0, -1].isnan()
    # every group but one below: its experts in order
    x = torch.zeros(2, 32)
    x[1, 24:] = 1.0
    _, e = binding.route_experts(x.cuda(), 3, groups=4, top_groups=1, score="sigmoid")
    assert e.tolist() == [[0, 1, 2], [24, 25, 26]]


def test_route_strided_rows():
    big = torch.randn(30, 100, device="cuda")
    for a, b in zip(binding.route_experts(big[:, 5:69], 6), binding.route_experts(big[:, 5:69].contiguous(), 6)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k,score", [(1, 1, 1, "softmax"), (9, 8, 3, "softmax"), (65, 100, 8, "softmax"),
                                         (33, 60, 5, "sigmoid"), (20, 300, 8, "softmax"), (5, 16, 16, "sigmoid")])
def test_route_backward_is_the_formula(T, E, k, score, renormalize, dtype):
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn(T, E, generator=g).to(dtype).cuda()
    gw = torch.randn(T, k, generator=g).cuda()
    _, experts = binding.route_experts(x, k, score=score, renormalize=renormalize, scale=1.5)
    got = binding.route_experts_backward(gw, x, experts, score=score, renormalize=renormalize, scale=1.5)
    x64 = x.double().requires_grad_(True)
    s = torch.softmax(x64, -1) if score == "softmax" else torch.sigmoid(x64)
    w = s.gather(1, experts.long())
    w = 1.5 * (w / w.sum(-1, keepdim=True) if renormalize else w)
    want = torch.autograd.grad(w, x64, gw.double())[0]
    # terms of the gradient: up to |g| * 1.5 each, a few dozen roundings of them; a term
    # divided by the sum of the chosen scores is weighted by those scores again
    size = 1.5 * gw.abs().double().sum(-1, keepdim=True)
    tol = 32 * EPS * size * s.detach().clamp(min=1e-3) / (w.detach().sum(-1, keepdim=True) / 1.5 if renormalize else 1)
    err = (got.double() - want).abs()
    assert bool((err <= tol + HALF_ULP[dtype] * want.abs()).all()), (err / tol).max()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward_is_the_difference(score):
    """Central differences of <g, weights> with the choice held: h = 2^-6, error
    h^2 / 6 of the third derivative (below 2 for these scores and k = 3 weights)
    and 2^-23 * |g| / h of rounding: 1e-3 together."""
    T, E, k, h = 1, 12, 3, 2.0 ** -6
    x = torch.linspace(-1, 1, E)[torch.randperm(E, generator=torch.Generator().manual_seed(2))].view(1, E)
    gw = torch.tensor([[0.7, -1.1, 0.4]]).cuda()
    w, experts = binding.route_experts(x.cuda(), k, score=score)
    got = binding.route_experts_backward(gw, x.cuda(), experts, score=score)

    def f(v):
        w_, e_ = binding.route_experts(v.cuda(), k, score=score)
        assert torch.equal(e_, experts)  # steps of h do not change the choice
        return (gw * w_).double().sum().item()

    for e in range(E):
        up, down = x.clone(), x.clone()
        up[0, e] += h
        down[0, e] -= h
        assert abs((f(up) - f(down)) / (2 * h) - got[0, e].item()) <= 1e-3


def test_route_backward_leaves_out_absent_slots():
    x = torch.randn(4, 10, device="cuda")
    experts = torch.tensor([[1, 2], [-1, 3], [10, -5], [0, 9]], dtype=torch.int32, device="cuda")
    gw = torch.ones(4, 2, device="cuda")
    got = binding.route_experts_backward(gw, x, experts, renormalize=False)
    s = torch.softmax(x.double(), -1)
    d = torch.zeros(4, 10, dtype=torch.float64, device="cuda")
    for t in range(4):
        for e in experts[t].tolist():
            if 0 <= e < 10:
                d[t, e] += 1
    want = s * (d - (d * s).sum(-1, keepdim=True))
    assert (got.double() - want).abs().max().item() <= 32 * EPS


def layout_of(experts, E):
    flat = experts.reshape(-1)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    counts = np.bincount(key, minlength=E + 1)
    return np.concatenate([[0], counts.cumsum()]), order, counts


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (7, 3, 5), (33, 1, 1024), (1000, 4, 33), (4097, 1, 16),
                                   (3000, 8, 256), (2731, 6, 1024), (16384, 4, 7), (70000, 2, 100)])
def test_layout(T, k, E):
    g = torch.Generator().manual_seed(T)
    experts = torch.randint(-1 if T % 2 else 0, E + (1 if T % 3 == 0 else 0), (T, k), generator=g, dtype=torch.int32)
    got = binding.experts_layout(experts.cuda(), E)
    offsets, order, counts = layout_of(experts.numpy(), E)
    data = got.data.cpu().numpy()
    assert np.array_equal(data[: E + 2], offsets)
    assert np.array_equal(got.offsets.cpu().numpy(), offsets[: E + 1])
    assert np.array_equal(got.order.cpu().numpy(), order)
    starts = np.concatenate([[0], (-(-counts[:E] // 128) * 128).cumsum()])
    assert np.array_equal(data[E + 2: 2 * E + 3], starts)
    dest = data[2 * E + 3 + T * k: 2 * E + 3 + 2 * T * k]
    key = np.where((experts.reshape(-1) >= 0) & (experts.reshape(-1) < E), experts.reshape(-1), E)
    place = np.empty(T * k, dtype=np.int64)
    place[order] = np.arange(T * k)
    want = np.where(key < E, starts[np.minimum(key, E)] + place - offsets[key], -1)
    assert np.array_equal(dest, want)
    wide = data[2 * E + 3 + 2 * T * k: 2 * E + 3 + 3 * T * k]
    want = np.where(key < E, starts[np.minimum(key, E)] // 128 * 224 + place - offsets[key], -1)
    assert np.array_equal(wide, want)


def test_layout_one_expert_and_none():
    for value in (3, -1, 9):
        experts = torch.full((500, 2), value, dtype=torch.int32)
        got = binding.experts_layout(experts.cuda(), 9)
        offsets, order, _ = layout_of(experts.numpy(), 9)
        assert np.array_equal(got.offsets.cpu().numpy(), offsets[:10]) and np.array_equal(got.order.cpu().numpy(), order)
    got = binding.experts_layout(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 9)
    assert got.offsets.cpu().tolist() == [0] * 10 and got.order.numel() == 0


def some_experts(seed, T, k, E, absent=False):
    g = torch.Generator().manual_seed(seed)
    e = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    if absent:
        e[torch.rand(T, k, generator=g) < 0.2] = -1
    return e.cuda()


EXPERTS = [(1, 1, 1, 1, 1), (1, 4, 16, 130, 100), (9, 2, 3, 64, 257), (70, 3, 5, 200, 96), (40, 8, 64, 129, 320),
           (300, 4, 7, 260, 64), (500, 2, 2, 128, 600), (700, 1, 2, 300, 129), (130, 6, 8, 100, 1000),
           (2, 2, 4, 200, 4100), (3, 4, 16, 1024, 4096), (1, 8, 64, 2100, 520), (1, 2, 4, 40, 9000)]


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("absent", [False, True])
@pytest.mark.parametrize("T,k,E,N,K", EXPERTS)
def test_experts_linear(T, k, E, N, K, absent, per_slot):
    experts = some_experts(T, T, k, E, absent)
    x, w = spread(1, T * k if per_slot else T, K), spread(2, E * N, K).view(E, N, K)
    bias = spread(3, E, N)
    layout = binding.experts_layout(experts, E)
    got = binding.experts_linear_mxfp4(x, binding.quantize_mxfp4(w), layout, bias, relu=True)
    xq, flat = mx_blocks(f64(x))[0], experts.reshape(-1).cpu().numpy()
    y, s = np.zeros((T * k, N)), np.zeros((T * k, N))
    for e in range(E):
        at = np.nonzero(flat == e)[0]
        y[at], s[at] = product_case(xq[at if per_slot else at // k], mx_blocks(f64(w[e]))[0], f64(bias[e]), True)
    check(got, y, s, K)
    assert (f64(got)[flat < 0] == 0).all()
    assert binding.check_device_error() == binding.IMC_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_experts_linear_types(dtype):
    T, k, E, N, K = 50, 3, 6, 140, 200
    experts = some_experts(5, T, k, E)
    x, w = spread(1, T, K + 8, dtype)[:, 8:], spread(2, E * N, K).view(E, N, K) / 16
    layout = binding.experts_layout(experts, E)
    wq = binding.quantize_mxfp4(w)
    got = binding.experts_linear_mxfp4(x, wq, layout)
    assert got.dtype == dtype
    xq, flat = mx_blocks(f64(x))[0], experts.reshape(-1).cpu().numpy()
    y, s = np.zeros((T * k, N)), np.zeros((T * k, N))
    for e in range(E):
        at = np.nonzero(flat == e)[0]
        y[at], s[at] = product_case(xq[at // k], mx_blocks(f64(w[e]))[0])
    check(got, y, s, K, dtype)
    wide = binding.experts_linear_mxfp4(x, wq, layout, out_dtype=torch.float32)
    assert torch.equal(wide.to(dtype), got)


@pytest.mark.parametrize("count", [1, 31, 33, 100, 129, 400])
def test_experts_linear_one_expert_has_all(count):
    E, N, K = 40, 130, 192
    experts = torch.full((count, 1), 17, dtype=torch.int32, device="cuda")
    x, w = spread(1, count, K), spread(2, E * N, K).view(E, N, K)
    got = binding.experts_linear_mxfp4(x, binding.quantize_mxfp4(w), binding.experts_layout(experts, E))
    y, s = product_case(mx_blocks(f64(x))[0], mx_blocks(f64(w[17]))[0])
    check(got, y, s, K)


def test_experts_linear_empty():
    experts = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    w = binding.quantize_mxfp4(spread(2, 80, 64).view(4, 20, 64))
    got = binding.experts_linear_mxfp4(torch.empty(0, 64, device="cuda"), w, binding.experts_layout(experts, 4))
    assert got.shape == (0, 20)
    none = torch.full((6, 2), -1, dtype=torch.int32, device="cuda")
    got = binding.experts_linear_mxfp4(spread(1, 6, 64), w, binding.experts_layout(none, 4))
    assert got.shape == (12, 20) and bool((got == 0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("per_slot,absent", [(False, False), (True, True), (False, True)])
@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 1, 1), (9, 2, 3, 64, 257), (70, 3, 5, 200, 96), (40, 8, 64, 129, 33),
                                       (500, 2, 2, 300, 600), (700, 1, 3, 257, 130)])
def test_experts_linear_backward_is_the_formula(T, k, E, N, K, per_slot, absent, dtype):
    experts = some_experts(T + 1, T, k, E, absent)
    layout = binding.experts_layout(experts, E)
    grad, x = spread(1, T * k, N, dtype), spread(2, T * k if per_slot else T, K, dtype)
    w = spread(3, E * N, K, dtype).view(E, N, K)
    gx, gw = binding.experts_linear_mxfp4_backward(grad, x, w, layout)
    flat, g64, x64 = experts.reshape(-1).cpu().numpy(), f64(grad), f64(x)
    y, s = np.zeros((T * k, K)), np.zeros((T * k, K))
    gq = mx_blocks(g64)[0]
    for e in range(E):
        at = np.nonzero(flat == e)[0]
        if len(at) == 0:
            assert bool((gw[e] == 0).all())
            continue
        y[at], s[at] = product_case(gq[at], mx_blocks(f64(w[e]).T)[0])
        want, size = product_case(mx_blocks(g64[at].T)[0], mx_blocks(x64[at if per_slot else at // k].T)[0])
        check(gw[e], want, size, len(at), dtype)
    if per_slot:
        check(gx, y, s, N, dtype)
    else:  # each slot's product is rounded to the type, then the slots are summed
        y3, s3 = y.reshape(T, k, K), s.reshape(T, k, K)
        tol = ((N / 64 + 2) * 2.0 ** -23 * s3 + HALF_ULP[dtype] * np.abs(y3)).sum(1)
        tol = 1.02 * tol + k * EPS * np.abs(y3).sum(1) + HALF_ULP[dtype] * np.abs(y3).sum(1)
        assert (np.abs(f64(gx) - y3.sum(1)) <= tol).all()
    assert binding.check_device_error() == binding.IMC_OK


def test_experts_linear_backward_is_the_difference():
    """On values that MXFP4 holds along both axes, gradients are exact differences."""
    T, k, E, N, K = 40, 2, 3, 32, 64
    g = torch.Generator().manual_seed(7)

    def values(rows, cols):
        v = torch.tensor([-4.0, -2.0, -1.0, 1.0, 2.0, 4.0])[torch.randint(0, 6, (rows, cols), generator=g)]
        v[::2, ::2] = 4.0  # a largest value in every block, whatever the order of the rows
        v[1::2, 1::2] = -4.0
        return v

    experts = some_experts(3, T, k, E)
    layout = binding.experts_layout(experts, E)
    x, grad = values(T, K).cuda(), values(T * k, N).cuda()
    w = values(E * N, K).view(E, N, K).cuda()
    gx, gw = binding.experts_linear_mxfp4_backward(grad, x, w, layout)

    def f(x_, w_):
        y = binding.experts_linear_mxfp4(x_, binding.quantize_mxfp4(w_), layout)
        return (grad.double() * y.double()).sum().item()

    base = f(x, w)
    for i, j in ((0, 1), (17, 4), (39, 62)):
        x2 = x.clone()
        x2[i, j] = 3.0
        assert f(x2, w) - base == gx[i, j].item() * (3.0 - x[i, j].item())
    for e, i, j in ((0, 0, 1), (1, 31, 62), (2, 6, 33)):
        w2 = w.clone()
        w2[e, i, j] = -3.0
        assert f(x, w2) - base == gw[e, i, j].item() * (-3.0 - w[e, i, j].item())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 8, 2048), (33, 3, 7), (100, 5, 129), (300, 8, 512), (9, 32, 40)])
def test_combine_and_gradients(T, k, N, dtype):
    y, w, grad = spread(1, T * k, N, dtype), torch.rand(T, k, device="cuda"), spread(3, T, N, dtype)
    y64, w64, g64 = f64(y).reshape(T, k, N), f64(w)[..., None], f64(grad)[:, None]
    want, size = (w64 * y64).sum(1), np.abs(w64 * y64).sum(1)
    got = f64(binding.experts_combine(y, w))
    tiny = 2.0 ** -24 if dtype == torch.float16 else 0.0
    assert (np.abs(got - want) <= k * EPS / 2 * size + HALF_ULP[dtype] * np.abs(want) * 1.01 + tiny).all()
    gy, gw = binding.experts_combine_backward(grad, y, w)
    want = (w64 * g64).reshape(T * k, N)
    assert (np.abs(f64(gy) - want) <= HALF_ULP[dtype] * np.abs(want) * 1.01 + EPS * np.abs(want) + tiny).all()
    want, size = (g64 * y64).sum(-1), np.abs(g64 * y64).sum(-1)
    assert (np.abs(f64(gw) - want) <= (N / 32 + 8) * EPS / 2 * size).all()


def test_combine_gradients_are_the_differences():
    """The sum is linear in y and in the weights: on small whole numbers its
    differences are exact."""
    T, k, N = 3, 4, 20
    g = torch.Generator().manual_seed(1)
    y = torch.randint(-4, 5, (T * k, N), generator=g).float().cuda()
    w = torch.randint(-3, 4, (T, k), generator=g).float().cuda()
    grad = torch.randint(-4, 5, (T, N), generator=g).float().cuda()
    gy, gw = binding.experts_combine_backward(grad, y, w)

    def f(y_, w_):
        return (grad.double() * binding.experts_combine(y_, w_).double()).sum().item()

    base = f(y, w)
    for i, j in ((0, 0), (5, 7), (11, 19)):
        y2 = y.clone()
        y2[i, j] += 2
        assert f(y2, w) - base == 2 * gy[i, j].item()
    for i, j in ((0, 0), (1, 3), (2, 2)):
        w2 = w.clone()
        w2[i, j] += 1
        assert f(y, w2) - base == gw[i, j].item()


def test_experts_block_in_a_graph():
    """Router logits to weighted sum, captured once and replayed on new tokens."""
    T, E, k, D, H = 24, 8, 2, 96, 160
    wr = spread(1, E, D) / 8
    w1 = binding.quantize_mxfp4(spread(2, E * H, D).view(E, H, D))
    w2 = binding.quantize_mxfp4(spread(3, E * D, H).view(E, D, H))

    def block(x):
        weights, experts = binding.route_experts(binding.linear(x, wr), k)
        layout = binding.experts_layout(experts, E)
        h = binding.experts_linear_mxfp4(x, w1, layout, relu=True)
        return binding.experts_combine(binding.experts_linear_mxfp4(h, w2, layout), weights)

    x = spread(4, T, D)
    want = block(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(x)
    graph.replay()
    assert torch.equal(out, want)
    x.copy_(spread(5, T, D))
    want = block(x)
    graph.replay()
    assert torch.equal(out, want)
