"""MXFP4 quantisation and products against their definition in 64 bits.

Tolerances.  Quantisation and dequantisation to fp32 / bf16 are exact.  A
product's terms are exact; its sum is rounded at most once per 64 values of K
(fp32 accumulator, one MMA at a time, possibly truncating: 2^-23 of the largest
partial sum, which sum|a b| bounds), once more for the bias, and once to the
output's type.
"""
import random

import numpy as np
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding

pytestmark = pytest.mark.gpu

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def mx_blocks(x):
    """(values MXFP4 holds for x, scale bytes, codes) by the definition, numpy float64."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    blocks = -(-cols // 32)
    y = np.zeros((rows, blocks * 32))
    y[:, :cols] = x
    y = y.reshape(rows, blocks, 32)
    bad = ~np.isfinite(y).all(-1)
    safe = np.where(np.isfinite(y), y, 0.0)
    top = np.abs(safe).max(-1)
    _, e = np.frexp(top)  # top = m * 2^e, 1/2 <= m < 1
    e = np.where(top > 0, np.clip(e - 1 - 2, -127, 127), -127)
    v = np.abs(np.ldexp(safe, -e[..., None]))
    # the nearest level; of two equally near ones the even code
    d = np.abs(v[..., None] - LEVELS)
    best = d.min(-1, keepdims=True)
    near = d == best
    code = np.where(near[..., ::2].any(-1), 2 * near[..., ::2].argmax(-1),
                    2 * near[..., 1::2].argmax(-1) + 1)
    code = np.where(near.sum(-1) == 1, near.argmax(-1), code)
    out = np.ldexp(np.copysign(LEVELS[code], safe), e[..., None])
    out[bad] = np.nan
    code = np.where(bad[..., None], 0, code + 8 * np.signbit(safe))
    scale = np.where(bad, 255, e + 127)
    return out.reshape(rows, -1)[:, :cols], scale.astype(np.uint8), code.reshape(rows, -1)


def f64(t):
    return t.detach().double().cpu().numpy()


def spread(seed, rows, cols, dtype=torch.float32):
    """Normal values whose blocks differ in size by several powers of two."""
    g = torch.Generator().manual_seed(seed)
    size = torch.exp2(torch.randint(-6, 7, (rows, cols), generator=g).float() / 2)
    return (torch.randn(rows, cols, generator=g) * size).to(dtype).cuda()


SHAPES = [(1, 1), (1, 31), (3, 32), (2, 33), (1, 4096), (127, 65), (129, 129), (300, 1000), (33, 96)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_is_the_definition(rows, cols, dtype):
    x = spread(rows * 1000 + cols, rows, cols, dtype)
    want, _, _ = mx_blocks(f64(x))
    assert np.array_equal(f64(binding.dequantize_mxfp4(binding.quantize_mxfp4(x))), want)
    want, _, _ = mx_blocks(f64(x).T)
    q = binding.quantize_mxfp4(x, transpose=True)
    assert q.shape == (cols, rows)
    assert np.array_equal(f64(binding.dequantize_mxfp4(q)), want)


def test_storage_is_as_documented():
    rows, cols = 150, 300
    x = spread(5, rows, cols)
    _, scale, code = mx_blocks(f64(x))
    data = binding.quantize_mxfp4(x).data.cpu().numpy()
    blocks = -(-cols // 32)
    pitch = 16 * blocks
    got = data[: rows * pitch].reshape(rows, pitch)
    assert np.array_equal(got & 15, code[:, 0::2]) and np.array_equal(got >> 4, code[:, 1::2])
    off = -(-rows * pitch // 512) * 512
    atoms = -(-blocks // 4)
    for r in range(rows):
        for b in range(blocks):
            at = off + ((r // 128) * atoms + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
            assert data[at] == scale[r, b], (r, b)
    assert data.size == binding.mxfp4_bytes(1, rows, cols)


@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_special_values(transpose):
    x = torch.zeros(12, 32)
    x[0] = 0.0
    x[1, 5] = float("inf")
    x[2, 5] = float("nan")
    x[3, :] = 1e-45                      # the smallest denormal
    x[4, :] = torch.finfo(torch.float32).max
    x[5, :] = -torch.finfo(torch.float32).max
    halves = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 7.99, 4.0]
    x[6, :10] = torch.tensor(halves)     # halfway cases; above 6
    x[7, :10] = -torch.tensor(halves)
    x[8, :10] = torch.tensor(halves) * 2.0 ** -126
    x[9, 0], x[9, 1] = 1e30, 1e-30       # a value lost beside a large one
    x[10, 3] = -float("inf")
    x[11, :] = torch.linspace(-6.5, 6.5, 32)
    want, _, _ = mx_blocks(x.double().numpy())
    src = x.cuda()
    q = (binding.quantize_mxfp4(src.t().contiguous(), transpose=True) if transpose
         else binding.quantize_mxfp4(src))
    assert np.array_equal(f64(binding.dequantize_mxfp4(q)), want, equal_nan=True)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_quantize_every_16_bit_value(dtype, transpose):
    """Each of the 65536 values, beside 31 others of its size and beside a large one."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = torch.cat([bits, bits.view(2048, 32).t().reshape(-1)]).view(4096, 32).view(dtype)
    want, _, _ = mx_blocks(x.double().numpy())
    src = x.t().contiguous().cuda() if transpose else x.cuda()
    got = binding.dequantize_mxfp4(binding.quantize_mxfp4(src, transpose=transpose))
    assert np.array_equal(f64(got), want, equal_nan=True)


@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_strides_and_batches(transpose):
    big = spread(3, 3 * 50, 201)
    for view in (big[:50, 1:98], big[5::3, :64], big[:1, 3:100], big[:, 8:72]):
        want, _, _ = mx_blocks(f64(view).T if transpose else f64(view))
        got = binding.dequantize_mxfp4(binding.quantize_mxfp4(view, transpose=transpose))
        assert np.array_equal(f64(got), want)
    w = big.view(3, 50, 201)[:, :, :70]
    got = f64(binding.dequantize_mxfp4(binding.quantize_mxfp4(w, transpose=transpose)))
    for e in range(3):
        want, _, _ = mx_blocks(f64(w[e]).T if transpose else f64(w[e]))
        assert np.array_equal(got[e], want)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("stride", [160, 168, 164, 162, 161])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_row_alignments(dtype, stride, transpose):
    """Rows that begin at multiples of 64, 32, 16, 8 and fewer bytes, whole and at an offset."""
    big = spread(stride, 133, stride, dtype)
    for view in (big[:, :160], big[:, 8:160], big[:, 4:132]):
        want, _, _ = mx_blocks(f64(view).T if transpose else f64(view))
        got = binding.dequantize_mxfp4(binding.quantize_mxfp4(view, transpose=transpose))
        assert np.array_equal(f64(got), want)


@pytest.mark.parametrize("M,N,K", [(130, 264, 160), (257, 132, 72), (64, 128, 128), (385, 130, 33)])
@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_is_quantised_both_ways(M, N, K, dtype):
    """Against the gradients of the operands quantised one by one: the same products."""
    dy, x, w = spread(6, M, N, dtype), spread(7, M, K, dtype), spread(8, N, K, dtype)
    dx, dw = binding.linear_mxfp4_backward(dy, x, w)
    t = lambda v: binding.quantize_mxfp4(v, transpose=True)  # noqa: E731
    assert torch.equal(dx, binding.linear_mxfp4(dy, t(w)))
    assert torch.equal(dw, binding.linear_mxfp4(t(dy), t(x), out_dtype=dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize_types(dtype):
    x = spread(9, 65, 77)
    want, _, _ = mx_blocks(f64(x))
    got = binding.dequantize_mxfp4(binding.quantize_mxfp4(x), dtype=dtype)
    assert got.dtype == dtype
    assert np.array_equal(f64(got), f64(torch.from_numpy(want).to(dtype)))


def product_case(x, w, bias=None, relu=False):
    """(exact result, sum of magnitudes) of the product of already quantised values."""
    y, s = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        y, s = y + bias, s + np.abs(bias)
    return (np.maximum(y, 0) if relu else y), s


HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def check(got, y, s, K, dtype=torch.float32):
    tol = (K / 64 + 2) * 2.0 ** -23 * s + HALF_ULP[dtype] * np.abs(y)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -24
    err = np.abs(f64(got) - y)
    assert (err <= tol).all(), f"worst {np.max(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"


MNK = [(1, 1, 1), (1, 129, 33), (2, 7, 64), (31, 128, 256), (32, 127, 257), (33, 64, 95),
       (64, 300, 130), (65, 128, 512), (127, 130, 1000), (128, 256, 63), (129, 100, 128),
       (255, 129, 320), (256, 1, 1056), (257, 257, 257), (700, 520, 2080), (1, 4096, 4096),
       (17, 1001, 1100), (513, 640, 4128), (2000, 1300, 160), (2100, 1100, 700), (4100, 515, 300),
       (1537, 2050, 1056), (3000, 2000, 31), (3, 40000, 700), (8, 20500, 2100), (5, 300, 6000)]


@pytest.mark.parametrize("M", [224 * 8, 224 * 9 + 1, 224 * 10 - 1, 256 * 8, 256 * 9 + 3])
@pytest.mark.parametrize("N,K", [(2100, 4096), (2048, 6144 + 32)])
def test_linear_tiles_of_224_tokens(M, N, K):
    """Sizes at which tokens quantised by the call are tiled otherwise than an operand
    quantised before: every output is the same sum."""
    x, w = spread(M, M, K, torch.bfloat16), binding.quantize_mxfp4(spread(N, N, K))
    assert torch.equal(binding.linear_mxfp4(x, w, out_dtype=torch.float32),
                       binding.linear_mxfp4(binding.quantize_mxfp4(x), w))
    assert binding.check_device_error() == binding.IMC_OK


@pytest.mark.parametrize("M,N,K", MNK)
def test_linear(M, N, K):
    x, w = spread(M + K, M, K), spread(N + K + 1, N, K)
    y, s = product_case(mx_blocks(f64(x))[0], mx_blocks(f64(w))[0])
    wq = binding.quantize_mxfp4(w)
    got = binding.linear_mxfp4(x, wq)
    check(got, y, s, K)
    # operands quantised before the call are the same operands
    assert torch.equal(got, binding.linear_mxfp4(binding.quantize_mxfp4(x), wq))
    assert torch.equal(got, binding.linear_mxfp4(x, w))
    assert binding.check_device_error() == binding.IMC_OK


@pytest.mark.parametrize("seed", range(24))
def test_linear_of_any_sizes(seed):
    r = random.Random(seed)
    M, N, K = (int(2 ** r.uniform(0, top)) for top in (11.5, 11, 12))
    x, w = spread(seed, M, K, torch.bfloat16), spread(seed + 1, N, K)
    y, s = product_case(mx_blocks(f64(x))[0], mx_blocks(f64(w))[0])
    check(binding.linear_mxfp4(x, w, out_dtype=torch.float32), y, s, K)
    assert binding.check_device_error() == binding.IMC_OK


@pytest.mark.parametrize("x_type", TYPES)
@pytest.mark.parametrize("out_type", TYPES)
@pytest.mark.parametrize("M", [3, 40, 100, 300])
def test_linear_types_bias_relu(M, x_type, out_type):
    N, K = 203, 420
    x, w = spread(M, M, K, x_type), spread(N, N, K) / 16
    bias = spread(77, 1, N)[0]
    y, s = product_case(mx_blocks(f64(x))[0], mx_blocks(f64(w))[0], f64(bias), relu=True)
    got = binding.linear_mxfp4(x, w, bias, relu=True, out_dtype=out_type)
    assert got.dtype == out_type
    check(got, y, s, K, out_type)


def test_linear_out_and_strided_rows():
    x, w = spread(1, 90, 300)[:, 4:260], spread(2, 70, 256)
    out = torch.full((90, 70), 7.0, device="cuda")
    got = binding.linear_mxfp4(x, w, out=out)
    assert got is out
    assert torch.equal(out, binding.linear_mxfp4(x.contiguous(), w))


@pytest.mark.parametrize("M", [5, 100, 300])
def test_linear_nan_stays_in_its_row_and_column(M):
    N, K = 140, 200
    x, w = spread(11, M, K), spread(12, N, K)
    ref = binding.linear_mxfp4(x, w)
    x[2, 50] = float("nan")
    w[130, 7] = float("inf")
    got = binding.linear_mxfp4(x, w)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[2], bad[:, 130] = True, True
    assert got[bad].isnan().all()
    assert torch.equal(got[~bad], ref[~bad])


def test_linear_long_rows():
    """K beyond the pipeline's depth many times, few rows: the sum over a long axis."""
    x, w = spread(21, 3, 65536), spread(22, 65, 65536)
    y, s = product_case(mx_blocks(f64(x))[0], mx_blocks(f64(w))[0])
    check(binding.linear_mxfp4(x, w), y, s, 65536)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (33, 65, 100), (200, 130, 96), (1000, 300, 513)])
def test_linear_backward_is_the_formula(M, N, K, dtype):
    dy, x, w = spread(1, M, N, dtype), spread(2, M, K, dtype), spread(3, N, K, dtype)
    dx, dw = binding.linear_mxfp4_backward(dy, x, w)
    mx = lambda v: mx_blocks(v)[0]  # noqa: E731
    y, s = product_case(mx(f64(dy)), mx(f64(w).T))
    check(dx, y, s, N, dtype)
    y, s = product_case(mx(f64(dy).T), mx(f64(x).T))
    check(dw, y, s, M, dtype)


@pytest.mark.parametrize("M,N,K", [(77, 130, 96), (700, 513, 2100)])
@pytest.mark.parametrize("dtype", TYPES)
def test_one_gradient_alone_is_the_same(M, N, K, dtype):
    """The C entry point without grad_x, and without grad_w (whose other input may be null)."""
    dy, x, w = spread(1, M, N, dtype), spread(2, M, K, dtype), spread(3, N, K, dtype)
    dx, dw = binding.linear_mxfp4_backward(dy, x, w)
    dx1, dw1 = torch.empty_like(dx), torch.empty_like(dw)
    dt = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[dtype]
    s = torch.cuda.current_stream().cuda_stream
    assert binding.mxfp4_linear_backward(dy.data_ptr(), None, w.data_ptr(), dt, M, N, K,
                                         dx1.data_ptr(), None, None, 0, s) == 0
    assert binding.mxfp4_linear_backward(dy.data_ptr(), x.data_ptr(), None, dt, M, N, K, None,
                                         dw1.data_ptr(), None, 0, s) == 0
    assert torch.equal(dx, dx1) and torch.equal(dw, dw1)


def test_linear_backward_is_the_difference():
    """On values that MXFP4 holds exactly along both axes, the gradients are the
    exact differences of <dy, linear(x, w)> (a step from one such value to another)."""
    M, N, K = 70, 40, 64
    g = torch.Generator().manual_seed(4)

    def values(rows, cols):
        v = torch.tensor([-4.0, -2.0, -1.0, 1.0, 2.0, 4.0])[torch.randint(0, 6, (rows, cols), generator=g)]
        v[::16, :], v[:, ::16] = 4.0, 4.0  # the largest value in every block: one scale for all
        return v.cuda()

    x, w, dy = values(M, K), values(N, K), values(M, N)
    dx, dw = binding.linear_mxfp4_backward(dy, x, w)

    def f(x_, w_):
        return (dy.double() * binding.linear_mxfp4(x_, w_).double()).sum().item()

    base = f(x, w)
    for i, j in ((1, 1), (17, 5), (69, 63), (3, 33)):
        x2 = x.clone()
        x2[i, j] = 3.0
        assert f(x2, w) - base == dx[i, j].item() * (3.0 - x[i, j].item())
    for i, j in ((1, 2), (39, 63), (7, 31)):
        w2 = w.clone()
        w2[i, j] = -3.0
        assert f(x, w2) - base == dw[i, j].item() * (-3.0 - w[i, j].item())


def test_linear_empty():
    w = spread(2, 70, 256)
    assert binding.linear_mxfp4(torch.empty(0, 256, device="cuda"), w).shape == (0, 70)
    assert binding.linear_mxfp4(spread(1, 3, 256), torch.empty(0, 256, device="cuda")).shape == (3, 0)


def test_streams_and_graph_replay():
    """A call on another stream, and a captured one replayed on new data."""
    x, w = spread(1, 50, 320), binding.quantize_mxfp4(spread(2, 130, 320))
    want = binding.linear_mxfp4(x, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = binding.linear_mxfp4(x, w)
    side.synchronize()
    assert torch.equal(got, want)
    static, out = x.clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.linear_mxfp4(static, w, out=out)
    for seed in (5, 6):
        x2 = spread(seed, 50, 320)
        static.copy_(x2)
        graph.replay()
        assert torch.equal(out, binding.linear_mxfp4(x2, w))


def test_calls_back_to_back_share_memory():
    """Calls in a row that reuse one another's freed scratch and feed each other."""
    w1, w2 = spread(1, 256, 128), spread(2, 128, 256)
    q1, q2 = binding.quantize_mxfp4(w1), binding.quantize_mxfp4(w2)
    x0 = spread(3, 200, 128)
    x, alone = x0, x0
    for _ in range(6):
        x = binding.linear_mxfp4(binding.linear_mxfp4(x, q1) / 64, q2) / 64
        h = binding.linear_mxfp4(alone, q1) / 64
        torch.cuda.synchronize()
        alone = binding.linear_mxfp4(h, q2) / 64
        torch.cuda.synchronize()
    assert torch.equal(x, alone)
