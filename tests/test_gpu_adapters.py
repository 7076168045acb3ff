"""Low-rank adapters and their gradients against the formulas in 64 bits.

Tolerances.  h = x a^T (and g = grad b): the operands enter exactly (fp32 in three bf16
pieces: the products that are left out are below 3 * 2^-25 of |x a|), and up to three fp32
additions, possibly truncating, are made per 16 terms, with a few more where partial sums
are joined: c1 = (3 * ceil(K / 16) + 24) * 2^-23 of sum |x a|.  h is kept for the second
product to 2^-17 of its value (16-bit types) or 2^-23 (fp32), and that product adds up to six
times per 16 terms: c2 = that + (6 * ceil(n / 16) + 8) * 2^-23 of sum |h b|, n its terms.
Base and product are added in fp32 (2^-23 of both), and the result is rounded once.
"""
import random

import numpy as np
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
TINY = {torch.float32: 1e-37, torch.bfloat16: 1e-37, torch.float16: 2.0 ** -24}
EPS = 2.0 ** -23


def f64(t):
    return t.detach().double().cpu().numpy()


def c1(terms):
    return (3 * -(-terms // 16) + 24) * EPS


def c2(terms, dtype):
    return (EPS if dtype == torch.float32 else 2.0 ** -17) + (6 * -(-terms // 16) + 8) * EPS


class Case:
    def __init__(self, seed, T, L, r, K, N, dtype, which="mixed", use_scale=True, use_base=True):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, size=1.0):
            return (size * torch.randn(*shape, generator=g)).to(dtype).cuda()

        self.T, self.L, self.r, self.K, self.N, self.dtype = T, L, r, K, N, dtype
        self.x, self.grad = normal(T, K), normal(T, N)
        self.a, self.b = normal(L, r, K, size=K ** -0.5), normal(L, N, r, size=r ** -0.5)
        self.scale = (0.25 + 2 * torch.rand(L, generator=g)).cuda() if use_scale else None
        self.base = normal(T, N) if use_base else None
        self.base_x = normal(T, K) if use_base else None
        w = torch.randint(-1, L, (T,), generator=g)
        if which == "one":
            w = torch.full((T,), L - 1)
        elif which == "none":
            w = torch.full((T,), -1)
        elif which == "runs":
            w = w.sort().values
        elif which == "outside":  # numbers that are no adapter's, on both sides
            w = torch.where(w < 0, L + 5, w) - 7 * (torch.rand(T, generator=g) < 0.2).long()
        self.which = w.to(torch.int32).cuda()
        self.layout = binding.experts_layout(self.which[:, None].contiguous(), L)

    def rows(self, l):
        return np.flatnonzero(self.which.cpu().numpy() == l)

    def s(self, l):
        return 1.0 if self.scale is None else float(self.scale[l])

    def forward64(self):
        x, a, b = f64(self.x), f64(self.a), f64(self.b)
        out = np.zeros((self.T, self.N)) if self.base is None else f64(self.base)
        tol = 2 * EPS * np.abs(out)
        with np.errstate(invalid="ignore"):
            for l in range(self.L):
                at = self.rows(l)
                if len(at) == 0:
                    continue
                h = self.s(l) * x[at] @ a[l].T
                eh = c1(self.K) * self.s(l) * np.abs(x[at]) @ np.abs(a[l]).T
                d, size = h @ b[l].T, np.abs(h) @ np.abs(b[l]).T
                tol[at] += eh @ np.abs(b[l]).T + c2(self.r, self.dtype) * size + 2 * EPS * np.abs(d)
                out[at] += d
        return out, self.rounded(out, tol)

    def rounded(self, v, tol):
        return 1.01 * tol + torch.finfo(self.dtype).eps / 2 * (np.abs(v) + tol) + TINY[self.dtype]

    def backward64(self):
        x, a, b, d = f64(self.x), f64(self.a), f64(self.b), f64(self.grad)
        gx = np.zeros((self.T, self.K)) if self.base_x is None else f64(self.base_x)
        ga, gb = np.zeros(a.shape), np.zeros(b.shape)
        tx, ta, tb = 2 * EPS * np.abs(gx), np.zeros(a.shape), np.zeros(b.shape)
        for l in range(self.L):
            at = self.rows(l)
            if len(at) == 0:
                continue
            s, n = self.s(l), len(at)
            h, g = s * x[at] @ a[l].T, s * d[at] @ b[l]
            eh = c1(self.K) * s * np.abs(x[at]) @ np.abs(a[l]).T
            eg = c1(self.N) * s * np.abs(d[at]) @ np.abs(b[l])
            v = g @ a[l]
            tx[at] += eg @ np.abs(a[l]) + c2(self.r, self.dtype) * np.abs(g) @ np.abs(a[l]) + 2 * EPS * np.abs(v)
            gx[at] += v
            ga[l], gb[l] = g.T @ x[at], d[at].T @ h
            ta[l] = (eg + c2(n, self.dtype) * np.abs(g)).T @ np.abs(x[at])
            tb[l] = np.abs(d[at]).T @ (eh + c2(n, self.dtype) * np.abs(h))
        return [(v, self.rounded(v, t)) for v, t in ((gx, tx), (ga, ta), (gb, tb))]

    def forward(self, **kw):
        return binding.adapters_linear(self.x, self.a, self.b, self.layout, self.base, scale=self.scale, **kw)

    def backward(self):
        return binding.adapters_linear_backward(self.grad, self.x, self.a, self.b, self.layout, self.base_x,
                                                scale=self.scale)

    def check(self, backward=True):
        within(self.forward(), *self.forward64(), self.dtype)
        if backward:
            for got, (want, tol) in zip(self.backward(), self.backward64()):
                within(got, want, tol, self.dtype)
        assert binding.check_device_error(None) == binding.IMC_OK


def within(got, want, tol, dtype):
    assert got.dtype == dtype and tuple(got.shape) == want.shape
    off = np.abs(f64(got) - want)
    worst = np.unravel_index(np.argmax(off - tol), off.shape) if off.size else ()
    assert (off <= tol).all(), f"{worst}: off by {off[worst]}, allowed {tol[worst]}"


SIZES = [(1, 1, 1, 1, 1), (1, 8, 16, 256, 512), (2, 3, 3, 33, 70), (7, 2, 8, 1024, 100), (8, 1, 16, 72, 64),
         (9, 40, 4, 100, 257), (64, 64, 16, 520, 128), (127, 5, 33, 130, 96), (128, 1, 64, 64, 256),
         (129, 2, 16, 200, 136), (300, 7, 20, 257, 129), (300, 3, 128, 96, 160), (257, 4, 100, 320, 64),
         (1000, 33, 8, 128, 40), (70, 1024, 2, 16, 24)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,L,r,K,N", SIZES)
def test_adapters(T, L, r, K, N, dtype):
    Case(T + 3 * r, T, L, r, K, N, dtype).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", ["one", "none", "runs", "outside"])
@pytest.mark.parametrize("T", [5, 140, 600])
def test_who_has_which(T, which, dtype):
    """All rows one adapter's, no row any, one run of rows after the other, numbers outside."""
    Case(T, T, 6, 12, 192, 80, dtype, which=which).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [3, 200])
def test_without_base_and_scale(T, dtype):
    Case(T, T, 3, 16, 136, 144, dtype, use_scale=False, use_base=False).check()


@pytest.mark.parametrize("seed", range(24))
def test_any_sizes(seed):
    r = random.Random(seed)
    T, L = int(np.exp(r.uniform(0, 7.5))), int(np.exp(r.uniform(0, 4)))
    Case(seed, T, L, r.randint(1, 128 if seed % 4 == 0 else 40), r.randint(1, 700), r.randint(1, 700),
         TYPES[seed % 3], which=r.choice(["mixed", "one", "runs"])).check()


@pytest.mark.parametrize("dtype,T,r,K,N", [(torch.bfloat16, 1, 16, 4096, 4096), (torch.bfloat16, 1500, 32, 4096, 1032),
                                           (torch.float32, 700, 16, 2048, 1500), (torch.float16, 520, 64, 1100, 4096)])
def test_large(dtype, T, r, K, N):
    Case(T, T, 5, r, K, N, dtype, which="runs").check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [6, 150])
def test_strided_and_unaligned_rows(T, dtype):
    """x with rows apart and at an odd element, a and b one element into their buffers."""
    c = Case(11, T, 4, 8, 120, 72, dtype)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten()
        return flat[1:].view(t.shape)

    wide = torch.full((T, 131), float("nan"), dtype=dtype, device="cuda")
    wide[:, 3:123] = c.x
    c.x = wide[:, 3:123]
    c.a, c.b, c.base = shifted(c.a), shifted(c.b), shifted(c.base)
    out = shifted(torch.zeros_like(c.base))
    want = c.forward64()
    within(c.forward(), *want, dtype)
    within(c.forward(out=out), *want, dtype)
    c.x, c.grad, c.base_x = shifted(c.x.contiguous()), shifted(c.grad), shifted(c.base_x)
    for got, (v, tol) in zip(c.backward(), c.backward64()):
        within(got, v, tol, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [9, 333])
def test_in_place_leaves_other_rows_alone(T, dtype):
    """out = base: a row without an adapter keeps its bits, a NaN's payload too; the others
    are as with an output of their own."""
    c = Case(T + 1, T, 3, 16, 200, 96, dtype)
    none = (c.which < 0).nonzero().flatten()
    c.x[none] = float("nan")
    c.base[none] = float("nan")
    want = c.forward()
    assert torch.isnan(want[none].float()).all() and torch.isfinite(want[c.which >= 0].float()).all()
    kind = torch.int32 if dtype == torch.float32 else torch.int16
    before = c.base.view(kind).clone()
    got = c.forward(out=c.base)
    assert got is c.base
    assert torch.equal(got.view(kind)[none], before[none])
    assert torch.equal(got[c.which >= 0], want[c.which >= 0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [9, 333])
def test_non_finite_values_stay_in_their_row(T, dtype):
    """An infinity or a NaN in one row of x or grad reaches no other row, and no gradient of
    an adapter that the row does not have."""
    c = Case(T + 2, T, 3, 16, 200, 96, dtype, which="runs")
    good, good_back = c.forward(), c.backward()
    bad = int(c.rows(1)[0])
    c.x[bad, 5], c.grad[bad, 7] = float("inf"), float("nan")
    keep = torch.arange(T, device="cuda") != bad
    assert torch.equal(c.forward()[keep], good[keep])
    assert not torch.isfinite(c.forward()[bad].float()).any()
    gx, ga, gb = c.backward()
    assert torch.equal(gx[keep], good_back[0][keep])
    others = [0, 2]
    assert torch.equal(ga[others], good_back[1][others]) and torch.equal(gb[others], good_back[2][others])
    assert not torch.isfinite(ga[1, :, 5].float()).any() and not torch.isfinite(gb[1, 7].float()).any()


@pytest.mark.parametrize("T", [1, 40, 700])
def test_twice_the_same_bits(T):
    c = Case(5, T, 3, 24, 300, 500, torch.bfloat16, which="runs")
    first, second = [c.forward(), *c.backward()], [c.forward(), *c.backward()]
    assert all(torch.equal(p, q) for p, q in zip(first, second))


def test_gradients_against_differences():
    """The gradients of sum(out * grad) are the differences of it, in fp32 at small sizes."""
    c = Case(4, 6, 2, 3, 10, 12, torch.float32)
    d = f64(c.grad)
    grads = c.backward()
    for name, grad, base in (("x", grads[0], f64(c.base_x)), ("a", grads[1], 0), ("b", grads[2], 0)):
        t = getattr(c, name)
        kept = t.clone()
        want = np.zeros(t.numel())
        for i in range(t.numel()):
            ends = []
            for step in (2.0 ** -3, -2.0 ** -3):  # out is linear in each of them
                t.copy_(kept)
                t.view(-1)[i] += step
                ends.append((f64(c.forward()) * d).sum())
            want[i] = (ends[0] - ends[1]) / 2.0 ** -2
        t.copy_(kept)
        # the forward's error (1e-5 of values of some units, 72 of them) over the step
        assert np.abs(f64(grad) - base - want.reshape(grad.shape)).max() <= 1e-2


@pytest.mark.parametrize("T", [4, 260])
def test_streams_and_graph_replay(T):
    """A call on another stream, and captured ones replayed on new data beside eager calls."""
    c = Case(8, T, 3, 16, 256, 192, torch.bfloat16)
    want, want_back = c.forward(), c.backward()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, got_back = c.forward(), c.backward()
    side.synchronize()
    assert torch.equal(got, want) and all(torch.equal(p, q) for p, q in zip(got_back, want_back))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = [c.forward(), *c.backward()]
        graphs.append((graph, outs))
    other = Case(9, T, 3, 16, 256, 192, torch.bfloat16)
    c.x.copy_(other.x)
    c.grad.copy_(other.grad)
    c.layout.data.copy_(other.layout.data)
    c.which.copy_(other.which)
    eager = [c.forward(), *c.backward()]
    for graph, outs in graphs:
        graph.replay()
        again = [c.forward(), *c.backward()]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, eager))
        assert all(torch.equal(p, q) for p, q in zip(again, eager))


def test_empty_calls():
    c = Case(1, 3, 2, 4, 16, 8, torch.float32)
    none = torch.empty(0, 1, dtype=torch.int32, device="cuda")
    layout = binding.experts_layout(none, 2)
    x = torch.empty(0, 16, device="cuda")
    assert binding.adapters_linear(x, c.a, c.b, layout).shape == (0, 8)
    gx, ga, gb = binding.adapters_linear_backward(torch.empty(0, 8, device="cuda"), x, c.a, c.b, layout)
    assert gx.shape == (0, 16) and not ga.any() and not gb.any()
    b = torch.empty(2, 0, 4, device="cuda")
    assert binding.adapters_linear(c.x, c.a, b, c.layout).shape == (3, 0)
    gx, ga, gb = binding.adapters_linear_backward(torch.empty(3, 0, device="cuda"), c.x, c.a, b, c.layout, c.base_x)
    assert torch.equal(gx, c.base_x) and not ga.any() and gb.shape == (2, 0, 4)


def test_parts_of_the_gradients():
    """The C entry point computes the gradients that have a place."""
    c = Case(6, 150, 3, 16, 128, 96, torch.bfloat16)
    want = c.backward()
    dt = binding.BF16
    n = binding.lowrank_linear_backward_workspace_bytes(150, 16)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for keep in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)):
        outs = [torch.full_like(w, 7.0) for w in want]
        ptr = [o.data_ptr() if k else None for o, k in zip(outs, keep)]
        rc = binding.lowrank_linear_backward(c.grad.data_ptr(), c.x.data_ptr(), c.a.data_ptr(), c.b.data_ptr(), dt,
                                             c.scale.data_ptr(), c.layout.data.data_ptr(), c.base_x.data_ptr(), *ptr,
                                             150, 3, 16, 128, 96, ws.data_ptr(), n, None)
        torch.cuda.synchronize()
        assert rc == 0
        for o, w, k in zip(outs, want, keep):
            assert torch.equal(o, w) if k else bool((o == 7).all())


def test_refused_by_the_torch_level():
    c = Case(1, 6, 2, 4, 16, 8, torch.float32)
    call = binding.adapters_linear
    with pytest.raises(TypeError):
        call(c.x, c.a, c.b, c.which, c.base)
    with pytest.raises(ValueError):  # another type
        call(c.x, c.a.bfloat16(), c.b, c.layout)
    with pytest.raises(ValueError):
        call(c.x, c.a, c.b[:, :, :3], c.layout)
    with pytest.raises(ValueError):
        call(c.x, c.a, c.b, c.layout, c.base[:, :7])
    with pytest.raises(ValueError):
        call(c.x, c.a, c.b, c.layout, scale=c.scale[:1])
    with pytest.raises(ValueError):  # a layout of other rows or adapters
        call(c.x[:5], c.a, c.b, c.layout)
    with pytest.raises(ValueError):
        call(c.x, c.a, c.b, binding.experts_layout(c.which[:, None].contiguous(), 3))
    with pytest.raises(ValueError):
        call(c.x, c.a, c.b, binding.experts_layout(c.which.view(3, 2), 2))
    with pytest.raises(ValueError):
        call(c.x.t(), c.a, c.b, c.layout)
    with pytest.raises(binding.ImcError):  # out overlaps x
        call(c.x[:, :8], c.a[:, :, :8].contiguous(), c.b, c.layout, out=c.x.view(-1)[:48].view(6, 8))
    with pytest.raises(binding.ImcError):  # out overlaps base, but is not it
        whole = torch.zeros(7, 8, device="cuda")
        call(c.x, c.a, c.b, c.layout, whole[:6], out=whole[1:])
    with pytest.raises(binding.ImcError):  # rank above 128
        a = torch.zeros(2, 129, 16, device="cuda")
        call(c.x, a, torch.zeros(2, 8, 129, device="cuda"), c.layout)
    with pytest.raises(ValueError):
        binding.adapters_linear_backward(c.grad[:, :4], c.x, c.a, c.b, c.layout)


@pytest.mark.parametrize("rows", [[5000], [0, 3000, 0, 0, 1], [64, 64, 64, 64, 64, 64], [1] * 40, [2, 700, 63, 65, 0, 128, 1500, 9],
                                  [640, 0, 1], [127, 130], [65]])
@pytest.mark.parametrize("r", [8, 40, 128])
def test_gradients_of_unequal_adapters(rows, r):
    """Adapters whose rows fill several blocks' runs, parts of them or none, in any order."""
    L, T = len(rows), sum(rows) + 3
    c = Case(T + r, T, L, r, 264, 392, torch.bfloat16)
    which = torch.cat([torch.full((n,), l) for l, n in enumerate(rows)] + [torch.full((3,), -1)])
    for order in (torch.arange(T), torch.randperm(T, generator=torch.Generator().manual_seed(T))):
        c.which = which[order].to(torch.int32).cuda()
        c.layout = binding.experts_layout(c.which[:, None].contiguous(), L)
        for got, (want, tol) in zip(c.backward(), c.backward64()):
            within(got, want, tol, c.dtype)
    assert binding.check_device_error(None) == binding.IMC_OK
