"""Low-rank adapters at the sizes where the product takes tiles of 128 rows (more than
sixteen rows an adapter and T * r above 8192).  Formulas and tolerances are those of the
smaller sizes' tests."""
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding
from test_gpu_adapters import Case, TYPES, f64, within

pytestmark = pytest.mark.gpu

SIZES = [(513, 1, 16, 64, 128), (600, 7, 20, 257, 129), (700, 40, 13, 96, 200), (1500, 2, 128, 136, 72),
         (1100, 3, 65, 520, 264), (2100, 128, 5, 72, 40), (9000, 1, 1, 16, 8), (640, 16, 33, 130, 1),
         (777, 4, 100, 1, 96), (1024, 1, 64, 64, 256), (1025, 2, 48, 192, 320), (17000, 1024, 2, 24, 40)]


def shifted(t):
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    flat[1:] = t.flatten()
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,L,r,K,N", SIZES)
def test_sizes(T, L, r, K, N, dtype):
    c = Case(T + r, T, L, r, K, N, dtype, which="runs" if T % 2 else "mixed")
    c.check(backward=False)
    assert binding.lowrank_linear_workspace_bytes(T, L, r) > 0  # the form with tiles


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", ["one", "none", "runs", "outside"])
def test_who_has_which(which, dtype):
    Case(3, 900, 6, 24, 192, 144, dtype, which=which).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", ["runs", "mixed"])
def test_without_base_and_scale(which, dtype):
    Case(4, 800, 3, 16, 136, 272, dtype, which=which, use_scale=False, use_base=False).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("what", ["x", "a", "b", "base", "out", "all"])
def test_strided_and_unaligned_rows(what, dtype):
    """Each operand alone, and all, where 16-byte copies cannot reach it; x with rows apart."""
    c = Case(11, 900, 4, 16, 120, 72, dtype, which="runs")
    want = c.forward64()
    if what in ("x", "all"):
        wide = torch.full((900, 131), float("nan"), dtype=dtype, device="cuda")
        wide[:, 3:123] = c.x
        c.x = wide[:, 3:123]
    for name in ("a", "b", "base"):
        if what in (name, "all"):
            setattr(c, name, shifted(getattr(c, name)))
    out = torch.zeros_like(c.base)
    if what in ("out", "all"):
        out = shifted(out)
    within(c.forward(out=out), *want, dtype)
    c.x, c.grad, c.base_x = c.x.contiguous(), shifted(c.grad) if what in ("x", "all") else c.grad, c.base_x
    for got, (v, tol) in zip(c.backward(), c.backward64()):
        within(got, v, tol, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_apart_at_whole_units(dtype):
    """x's rows 16-byte aligned, with other values (NaN) between them."""
    c = Case(12, 700, 3, 16, 120, 136, dtype)
    wide = torch.full((700, 160), float("nan"), dtype=dtype, device="cuda")
    wide[:, 16:136] = c.x
    c.x = wide[:, 16:136]
    within(c.forward(), *c.forward64(), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", ["runs", "mixed"])
@pytest.mark.parametrize("N", [96, 257])
def test_in_place_leaves_other_rows_alone(N, which, dtype):
    c = Case(N, 1000, 3, 16, 200, N, dtype, which=which)
    none = (c.which < 0).nonzero().flatten()
    assert len(none) > 100
    c.x[none] = float("nan")
    c.base[none] = float("nan")
    want = c.forward()
    assert torch.isnan(want[none].float()).all() and torch.isfinite(want[c.which >= 0].float()).all()
    kind = torch.int32 if dtype == torch.float32 else torch.int16
    before = c.base.view(kind).clone()
    got = c.forward(out=c.base)
    assert torch.equal(got.view(kind)[none], before[none])
    assert torch.equal(got[c.which >= 0], want[c.which >= 0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", ["runs", "mixed"])
def test_non_finite_values_stay_in_their_row(which, dtype):
    c = Case(5, 1000, 3, 16, 200, 96, dtype, which=which)
    good, good_back = c.forward(), c.backward()
    bad = int(c.rows(1)[0])
    c.x[bad, 5], c.grad[bad, 7] = float("inf"), float("nan")
    keep = torch.arange(1000, device="cuda") != bad
    assert torch.equal(c.forward()[keep], good[keep])
    assert not torch.isfinite(c.forward()[bad].float()).any()
    gx, ga, gb = c.backward()
    assert torch.equal(gx[keep], good_back[0][keep])
    others = [0, 2]
    assert torch.equal(ga[others], good_back[1][others]) and torch.equal(gb[others], good_back[2][others])
    assert not torch.isfinite(ga[1, :, 5].float()).any() and not torch.isfinite(gb[1, 7].float()).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [12, 9000])
def test_an_infinity_beside_a_rank_that_is_padded(T, dtype):
    """Rank 1: an infinite x gives infinite outputs of the product's sign, not NaN."""
    c = Case(T, T, 1, 1, 32, 16, dtype, which="one", use_base=False)
    c.x[5, 3] = float("inf")
    got = f64(c.forward())[5]
    want = (c.scale[0] * torch.sign(c.a[0, 0, 3].float()) * torch.sign(c.b[0, :, 0].float())).cpu().double().numpy()
    assert (got == want * float("inf")).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", ["runs", "mixed"])
def test_twice_the_same_bits(which, dtype):
    c = Case(5, 1700, 3, 24, 304, 504, dtype, which=which)
    first, second = [c.forward(), *c.backward()], [c.forward(), *c.backward()]
    assert all(torch.equal(p, q) for p, q in zip(first, second))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_streams_at_once(dtype):
    """Calls of two streams that run beside each other, products and gradients, many and few rows."""
    cases = [Case(20, 900, 3, 16, 256, 512, dtype, which="runs"), Case(21, 40, 3, 16, 256, 512, dtype),
             Case(22, 1300, 8, 32, 128, 264, dtype)]
    want = [[c.forward(), *c.backward()] for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    for turn in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                c = (turn + i) % len(cases)
                got.append((c, [cases[c].forward(), *cases[c].backward()]))
    torch.cuda.synchronize()
    for c, outs in got:
        assert all(torch.equal(p, q) for p, q in zip(outs, want[c]))
    assert binding.check_device_error(None) == binding.IMC_OK


def test_graph_replays_with_other_adapters():
    """A captured call, layout included, replayed for other rows' numbers and data."""
    c = Case(8, 900, 5, 16, 256, 192, torch.bfloat16, which="runs")
    number = c.which[:, None].clone()
    c.forward()

    def step():
        c.layout = binding.experts_layout(number, 5)
        return [c.forward(), *c.backward()]

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    layout = c.layout
    for seed, which in ((9, "mixed"), (10, "one"), (11, "none")):
        other = Case(seed, 900, 5, 16, 256, 192, torch.bfloat16, which=which)
        number.copy_(other.which[:, None])
        c.x.copy_(other.x)
        c.grad.copy_(other.grad)
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, eager))
        c.layout = layout


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,L,r,K,N", [(1500, 1, 4, 72, 56), (1200, 75, 16, 96, 133), (1100, 70, 24, 200, 64),
                                       (2000, 130, 8, 64, 72), (256, 1, 32, 128, 96), (257, 1, 32, 128, 96),
                                       (272, 17, 100, 80, 40), (273, 17, 100, 80, 40)])
def test_around_the_rules_for_few_rows(T, L, r, K, N, dtype):
    Case(T + L, T, L, r, K, N, dtype).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,L,r,K,N,which", [(480, 10, 33, 100, 264, "one"), (480, 10, 16, 1028, 36, "mixed"),
                                             (481, 10, 16, 1028, 36, "mixed"), (160, 10, 5, 77, 91, "runs"),
                                             (161, 10, 5, 77, 91, "runs"), (40, 9, 128, 130, 8, "none"),
                                             (900, 60, 18, 515, 258, "outside")])
def test_gradients_of_adapters_with_few_rows(T, L, r, K, N, which, dtype):
    """Around the rules for the gradients' form: 48 rows an adapter, 16 where rows are not aligned."""
    c = Case(T, T, L, r, K, N, dtype, which=which)
    for got, (want, tol) in zip(c.backward(), c.backward64()):
        within(got, want, tol, dtype)
    assert binding.check_device_error(None) == binding.IMC_OK


def test_places_beyond_32_bits():
    """More than 2^31 elements of x, of out and of the gradients, checked at both ends."""
    T, wide, L, r, n = 270000, 8192, 3, 16, 64
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, size=1.0):
        return (size * torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16))

    which = torch.randint(-1, L, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    layout = binding.experts_layout(which, L)
    some = torch.cat([torch.arange(40), torch.arange(T - 40, T)]).cuda()
    l = which[some, 0]
    big, small = normal(T, wide), normal(T, n)
    wide_w, narrow_w = normal(L, r, wide, size=wide ** -0.5), normal(L, n, r, size=r ** -0.5)

    def close(got, want):
        # an output's rounding of 2^-9, and h's 2^-17 times the terms' sizes, some units beside it
        off = (got.double() - want).abs().max().item()
        assert off <= 2.0 ** -8 * want.abs().max().item(), off

    def plain(x, a, b, base):
        out = base[some].double()
        for i in range(L):
            mine = (l == i).double()[:, None]
            out += mine * (x[some].double() @ a[i].double().t() @ b[i].double().t())
        return out

    close(binding.adapters_linear(big, wide_w, narrow_w, layout, small)[some], plain(big, wide_w, narrow_w, small))
    up_a, up_b = normal(L, r, n, size=n ** -0.5), normal(L, wide, r, size=r ** -0.5)
    close(binding.adapters_linear(small, up_a, up_b, layout, big)[some], plain(small, up_a, up_b, big))
    gx, ga, gb = binding.adapters_linear_backward(big, small, up_a, up_b, layout, small)  # grad is wide
    close(gx[some], plain(big, up_b.transpose(1, 2).contiguous(), up_a.transpose(1, 2).contiguous(), small))
    rows = (which[:, 0] == 1).nonzero().flatten()
    h = small[rows].float() @ up_a[1].float().t()
    close(gb[1, -128:], big[rows, -128:].double().t() @ h.double())
    gx, ga, gb = binding.adapters_linear_backward(small, big, wide_w, narrow_w, layout, big)  # x is wide
    close(gx[some], plain(small, narrow_w.transpose(1, 2).contiguous(), wide_w.transpose(1, 2).contiguous(), big))
    close(ga[1, :, -128:], (small[rows].double() @ narrow_w[1].double()).t() @ big[rows, -128:].double())
    assert binding.check_device_error(None) == binding.IMC_OK


@pytest.mark.parametrize("L", [4, 40, 180])
@pytest.mark.parametrize("r", [33, 64, 65, 128])
def test_high_ranks_in_fp32(r, L):
    """Ranks whose operands leave two parts of base their room, or none; with and without a long table of adapters."""
    Case(r + L, 16 * L + 300, L, r, 72, 264, torch.float32, which="runs" if L == 4 else "mixed").check()
