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
