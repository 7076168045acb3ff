"""The 4-bit and expert operators at sizes that take their other kernels and tile forms,
against the definitions in 64 bits, which are computed on the GPU here (the sizes are
large).  Tolerances as in the tests of the small sizes."""
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding
from test_gpu_mxfp4 import HALF_ULP, TYPES, f64, mx_blocks

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -23


def power(n):
    """2^n in 64 bits, exactly."""
    return ((n.to(torch.int64) + 1023) << 52).view(torch.float64)


def held(x):
    """The values that MXFP4 holds for the rows of x, by the definition in 64 bits: a multiple
    of the step at the value's own power of two (.5 below 1), halfway cases to the even
    multiple (which has the even code), 6 at most."""
    x = x.double()
    cols = x.shape[-1]
    y = torch.nn.functional.pad(x, (0, -cols % 32)).unflatten(-1, (-1, 32))
    top = y.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, (torch.frexp(top).exponent - 3).clamp(-127, 127), -127)
    v = y * power(-e)
    step = power((torch.frexp(v).exponent - 1).clamp(min=0) - 1)
    v = ((v / step).round_() * step).clamp_(-6, 6)
    return (v * power(e)).flatten(-2)[..., :cols]


def spread(seed, *shape, dtype=torch.float32):
    """Normal values whose blocks differ in size by several powers of two."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = torch.exp2(torch.randint(-6, 7, shape, generator=g, device="cuda").float() / 2)
    return (torch.randn(shape, generator=g, device="cuda") * size).to(dtype)


def some_experts(seed, T, k, E, absent=0.0, unused=()):
    """k different experts a token, the first ones asked for more often; `absent` of the slots
    have none, the `unused` experts have no slot."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ask = 2 * torch.randn(T, E, generator=g, device="cuda") - 3 * torch.arange(E, device="cuda") / E
    ask[:, list(unused)] = -1e9
    e = ask.topk(k, -1).indices.to(torch.int32)
    e[torch.rand(T, k, generator=g, device="cuda") < absent] = -1
    return e


def check(got, y, s, K):
    """A product against its exact value y and the sum s of its terms' magnitudes."""
    tol = (K / 64 + 2) * EPS * s + HALF_ULP[got.dtype] * y.abs()
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -24
    err = (got.double() - y).abs()
    assert bool((err <= tol).all()), f"worst {(err / tol.clamp(min=1e-300)).max().item():.3g} of the tolerance"


def test_the_definition_is_the_definition():
    """held() and the other tests' definition, written apart."""
    for seed, rows, cols in ((1, 65, 97), (2, 300, 32)):
        x = spread(seed, rows, cols)
        x[::5] *= 2.0 ** -140
        x[1, :8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
        assert (f64(held(x)) == mx_blocks(f64(x))[0]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,N,K", [(40, 8, 16, 96, 200), (300, 6, 6, 130, 65), (700, 3, 4, 64, 128)])
def test_gradient_of_shared_rows_is_rounded_once(T, k, E, N, K, dtype):
    """A token's gradient is the fp32 sum of its slots' products, rounded to the type once."""
    experts = some_experts(T, T, k, E, absent=0.1)
    layout = binding.experts_layout(experts, E)
    grad, x, w = spread(1, T * k, N, dtype=dtype), spread(2, T, K, dtype=dtype), spread(3, E, N, K, dtype=dtype)
    gx, _ = binding.experts_linear_mxfp4_backward(grad, x, w, layout)
    assert gx.dtype == dtype
    g, flat = held(grad), experts.flatten()
    y, s = torch.zeros(T * k, K, dtype=torch.float64, device="cuda"), torch.zeros(T * k, K, dtype=torch.float64, device="cuda")
    for e in range(E):
        at, we = (flat == e).nonzero().flatten(), held(w[e].t())
        y[at], s[at] = g[at] @ we.t(), g[at].abs() @ we.abs().t()
    y, s = y.view(T, k, K), s.view(T, k, K).sum(1)
    # the products' sums, the sum of k of them (2^-24 of the magnitudes each), one rounding
    tol = (N / 64 + 2) * EPS * s + 1.02 * k * EPS / 2 * s + 1.02 * HALF_ULP[dtype] * y.sum(1).abs()
    tol = tol + (2.0 ** -24 if dtype == torch.float16 else 0)
    err = (gx.double() - y.sum(1)).abs()
    assert bool((err <= tol).all()), f"worst {(err / tol).max().item():.3g} of the tolerance"
    assert binding.check_device_error() == binding.IMC_OK


# Sizes beyond the tiles and blocks of the small tests: four blocks a lane and several tiles a
# CTA in the column quantiser, several rows a group in the row quantiser and its inverse.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(2500, 4100), (4999, 4101), (5120, 4104), (12800, 9600)])
def test_quantize_large(rows, cols, dtype):
    x = spread(rows + cols, rows, cols, dtype=dtype)
    want = held(x)
    q = binding.quantize_mxfp4(x)
    for out in TYPES:
        assert torch.equal(binding.dequantize_mxfp4(q, dtype=out), want.to(out))
    del want
    q = binding.quantize_mxfp4(x, transpose=True)
    assert torch.equal(binding.dequantize_mxfp4(q).double(), held(x.t()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols,first", [(4100, 0), (4096, 4), (4095, 1)])
def test_quantize_large_strided_batch(cols, first, dtype):
    big = spread(cols, 3, 2600, 4104, dtype=dtype)
    x = big[:, 50:2550, first:first + cols]
    for transpose in (False, True):
        q = binding.quantize_mxfp4(x, transpose=transpose)
        want = held(x.transpose(1, 2) if transpose else x)
        assert q.shape == tuple(want.shape)
        assert torch.equal(binding.dequantize_mxfp4(q).double(), want)


# K split over two, four and eight CTAs, with the tokens quantised by the product (up to 8)
# and before it (up to 32).
@pytest.mark.parametrize("K", [4200, 8300, 16500])
@pytest.mark.parametrize("M", [1, 8, 9, 17, 32])
def test_linear_split_over_k(M, K):
    x, w, bias = spread(M, M, K, dtype=torch.bfloat16), spread(K, 300, K), spread(3, 300)
    xq, wq = held(x), held(w)
    y, s = xq @ wq.t() + bias.double(), xq.abs() @ wq.abs().t() + bias.abs().double()
    packed = binding.quantize_mxfp4(w)
    for out in TYPES:
        got = binding.linear_mxfp4(x, packed, bias, relu=True, out_dtype=out)
        check(got, y.clamp(min=0), s, K)
    assert torch.equal(binding.linear_mxfp4(x, packed, out_dtype=torch.float32),
                       binding.linear_mxfp4(binding.quantize_mxfp4(x), packed))
    assert binding.check_device_error() == binding.IMC_OK


# Tiles of 224 tokens for both gradients, more of them than CTA pairs; one launch for w's and
# x's columns with four blocks a lane; and tiles of 256 for both.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(2500, 4100, 1100), (3500, 4100, 2100), (2048, 2040, 2300)])
def test_linear_backward_large(M, N, K, dtype):
    dy, x, w = spread(1, M, N, dtype=dtype), spread(2, M, K, dtype=dtype), spread(3, N, K, dtype=dtype)
    dx, dw = binding.linear_mxfp4_backward(dy, x, w)
    for got, a, b, depth in ((dx, held(dy), held(w.t()), N), (dw, held(dy.t()), held(x.t()), M)):
        check(got, a @ b.t(), a.abs() @ b.abs().t(), depth)
    # one gradient alone is the same
    dx1, dw1 = torch.empty_like(dx), torch.empty_like(dw)
    dt, s = binding._dtype_id(dtype, "dtype"), torch.cuda.current_stream().cuda_stream
    assert binding.mxfp4_linear_backward(dy.data_ptr(), None, w.data_ptr(), dt, M, N, K, dx1.data_ptr(),
                                         None, None, 0, s) == 0
    assert binding.mxfp4_linear_backward(dy.data_ptr(), x.data_ptr(), None, dt, M, N, K, None,
                                         dw1.data_ptr(), None, 0, s) == 0
    assert torch.equal(dx, dx1) and torch.equal(dw, dw1)
    assert binding.check_device_error() == binding.IMC_OK


# More tiles than CTA pairs, runs of different lengths, experts without rows between them.
UNEVEN = [(3000, 4, 16, 600, 2100, 0.0, ()), (2000, 3, 24, 300, 1100, 0.1, (0, 7, 8, 9, 23)), (900, 2, 40, 520, 700, 0.3, (3, 39))]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("T,k,E,N,K,absent,unused", UNEVEN)
def test_experts_large(T, k, E, N, K, absent, unused, per_slot, dtype):
    experts = some_experts(T, T, k, E, absent, unused)
    layout, flat = binding.experts_layout(experts, E), experts.flatten()
    x = spread(1, T * k if per_slot else T, K, dtype=dtype)
    w, grad = spread(2, E, N, K, dtype=dtype), spread(3, T * k, N, dtype=dtype)
    out = binding.experts_linear_mxfp4(x, binding.quantize_mxfp4(w), layout)
    gx, gw = binding.experts_linear_mxfp4_backward(grad, x, w, layout)
    assert bool((out[flat < 0] == 0).all())
    xq, gq = held(x), held(grad)
    dx = torch.zeros(T * k, K, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(dx)
    used = 0
    for e in range(E):
        at = (flat == e).nonzero().flatten()
        if len(at) == 0:
            assert bool((gw[e] == 0).all())
            continue
        used += 1
        row = at if per_slot else at // k
        wq, wt = held(w[e]), held(w[e].t())
        check(out[at], xq[row] @ wq.t(), xq[row].abs() @ wq.abs().t(), K)
        gc, xc = held(grad[at].t()), held(x[row].t())
        check(gw[e], gc @ xc.t(), gc.abs() @ xc.abs().t(), len(at))
        dx[at], size[at] = gq[at] @ wt.t(), gq[at].abs() @ wt.abs().t()
    assert used <= E - len(unused)
    if per_slot:
        check(gx, dx, size, N)
    else:
        y, s = dx.view(T, k, K).sum(1), size.view(T, k, K).sum(1)
        tol = (N / 64 + 2) * EPS * s + 1.02 * k * EPS / 2 * s + 1.02 * HALF_ULP[dtype] * y.abs()
        tol = tol + (2.0 ** -24 if dtype == torch.float16 else 0)
        assert bool(((gx.double() - y).abs() <= tol).all())
    assert binding.check_device_error() == binding.IMC_OK


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k,groups,top_groups", [(33, 1, 1, 1, 1), (19, 24, 3, 24, 4), (40, 32, 8, 32, 9)])
def test_route_types_of_single_experts(T, E, k, groups, top_groups, dtype):
    """Groups of one expert each, in every type (no bias, so equal logits are exact ties)."""
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(T)).to(dtype).cuda()
    w, experts = binding.route_experts(x, k, groups=groups, top_groups=top_groups)
    want = x.double().sort(dim=-1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(experts.long(), want)
    s = torch.softmax(x.double(), -1).gather(1, want)
    s = s / s.sum(-1, keepdim=True)
    assert bool(((w.double() - s).abs() <= 16 * EPS * s).all())


def test_calls_that_launch_nothing():
    """Empty gradients, and a matrix and a layout made from stored buffers."""
    for M, N in ((0, 70), (5, 0)):
        x, w = spread(1, M, 64), spread(2, N, 64)
        dx, dw = binding.linear_mxfp4_backward(binding.linear_mxfp4(x, w), x, w)
        assert dx.shape == (M, 64) and dw.shape == (N, 64) and bool((dx == 0).all()) and bool((dw == 0).all())
    x, w = spread(3, 40, 96), spread(4, 50, 96)
    stored = binding.quantize_mxfp4(w).data.cpu()
    q = binding.MxFp4(stored.cuda(), 1, 50, 96, False)
    assert torch.equal(binding.linear_mxfp4(x, q), binding.linear_mxfp4(x, w))
    with pytest.raises(ValueError):
        binding.dequantize_mxfp4(binding.MxFp4(stored, 1, 50, 96, False))  # still on the host
    with pytest.raises(ValueError):
        binding.linear_mxfp4(x, binding.MxFp4(stored, 1, 50, 96, False))
    layout = binding.experts_layout(some_experts(1, 40, 2, 5), 5)
    again = binding.ExpertsLayout(layout.data.clone(), 40, 2, 5)
    we = binding.quantize_mxfp4(spread(5, 5, 30, 96))
    assert torch.equal(binding.experts_linear_mxfp4(x, we, again), binding.experts_linear_mxfp4(x, we, layout))
