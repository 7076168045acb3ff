"""Refusals of the adapters' and the balance loss's entry points: every bad argument gets
its documented status before any CUDA call (fake, never dereferenced addresses), and a
well-formed call without a GPU fails loudly."""
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding, build
from test_boundary_host import without_gpu

P = [0x100000000 * i for i in range(1, 14)]
ARG, SHAPE, NULL, ALIAS = (binding.IMC_ERR_ARG, binding.IMC_ERR_SHAPE, binding.IMC_ERR_NULL,
                           binding.IMC_ERR_ALIAS)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def lowrank(x=P[0], dtype=0, ld=64, a=P[1], b=P[2], scale=P[3], layout=P[4], base=P[5], out=P[6], T=9000, L=3, r=8,
            K=64, N=32, ws=P[7], nbytes=1 << 22):
    return binding.lowrank_linear(x, dtype, ld, a, b, scale, layout, base, out, T, L, r, K, N, ws, nbytes, None)


def lowrank_back(grad=P[0], x=P[1], a=P[2], b=P[3], dtype=0, scale=P[4], layout=P[5], base=P[6], gx=P[7], ga=P[8],
                 gb=P[9], T=9, L=3, r=8, K=64, N=32, ws=P[10], nbytes=1 << 20):
    return binding.lowrank_linear_backward(grad, x, a, b, dtype, scale, layout, base, gx, ga, gb, T, L, r, K, N, ws,
                                           nbytes, None)


def balance(logits=P[0], dtype=0, T=9000, E=16, ld=16, experts=P[1], k=2, score=0, offsets=P[2], S=3, loss=P[3],
            counts=P[4], ws=P[5], nbytes=1 << 20):
    return binding.moe_balance(logits, dtype, T, E, ld, experts, k, score, offsets, S, loss, counts, ws, nbytes, None)


def balance_back(gl=P[0], logits=P[1], dtype=0, T=9, E=16, ld=16, experts=P[2], k=2, score=0, counts=P[3],
                 offsets=P[4], S=3, gw=P[5], renorm=1, scale=1.0, out=P[6]):
    return binding.moe_balance_backward(gl, logits, dtype, T, E, ld, experts, k, score, counts, offsets, S, gw, renorm,
                                        scale, out, None)


BAD = [
    (lowrank, dict(dtype=3), ARG), (lowrank, dict(T=-1), SHAPE), (lowrank, dict(T=2 ** 27 + 1), SHAPE),
    (lowrank, dict(L=0), SHAPE), (lowrank, dict(L=1025), SHAPE), (lowrank, dict(r=0), SHAPE),
    (lowrank, dict(r=129), SHAPE), (lowrank, dict(K=0), SHAPE), (lowrank, dict(N=-1), SHAPE),
    (lowrank, dict(K=2 ** 31, ld=2 ** 31), SHAPE), (lowrank, dict(ld=63), SHAPE), (lowrank, dict(x=None), NULL),
    (lowrank, dict(a=None), NULL), (lowrank, dict(b=None), NULL), (lowrank, dict(layout=None), NULL),
    (lowrank, dict(out=None), NULL), (lowrank, dict(x=P[0] + 2), ARG), (lowrank, dict(dtype=2, b=P[2] + 1), ARG),
    (lowrank, dict(scale=P[3] + 2), ARG), (lowrank, dict(layout=P[4] + 1), ARG), (lowrank, dict(base=P[5] + 2), ARG),
    (lowrank, dict(out=P[6] + 2), ARG), (lowrank, dict(out=P[0] + 4), ALIAS), (lowrank, dict(out=P[1]), ALIAS),
    (lowrank, dict(out=P[2]), ALIAS), (lowrank, dict(out=P[3]), ALIAS), (lowrank, dict(out=P[4]), ALIAS),
    (lowrank, dict(out=P[5] + 4), ALIAS), (lowrank, dict(out=P[5] - 4), ALIAS),
    (lowrank, dict(K=2 ** 20 + 1, ld=2 ** 20 + 1), SHAPE), (lowrank, dict(N=2 ** 20 + 1), SHAPE),
    (lowrank, dict(nbytes=64), ARG), (lowrank, dict(ws=P[7] + 8), ARG), (lowrank, dict(ws=P[0]), ALIAS),
    (lowrank, dict(ws=P[4]), ALIAS), (lowrank, dict(ws=P[5]), ALIAS), (lowrank, dict(ws=P[6]), ALIAS),
    (lowrank_back, dict(dtype=-1), ARG), (lowrank_back, dict(T=0), SHAPE), (lowrank_back, dict(N=0), SHAPE),
    (lowrank_back, dict(r=129), SHAPE), (lowrank_back, dict(L=0), SHAPE), (lowrank_back, dict(grad=None), NULL),
    (lowrank_back, dict(x=None), NULL), (lowrank_back, dict(a=None), NULL), (lowrank_back, dict(b=None), NULL),
    (lowrank_back, dict(layout=None), NULL), (lowrank_back, dict(gx=P[7] + 1), ARG),
    (lowrank_back, dict(ga=P[8] + 2), ARG), (lowrank_back, dict(gb=P[9] + 2), ARG),
    (lowrank_back, dict(base=P[6] + 2), ARG), (lowrank_back, dict(nbytes=8), ARG), (lowrank_back, dict(ws=P[10] + 4), ARG),
    (lowrank_back, dict(gx=P[0]), ALIAS), (lowrank_back, dict(gx=P[6] + 4), ALIAS), (lowrank_back, dict(ga=P[2]), ALIAS),
    (lowrank_back, dict(gb=P[3]), ALIAS), (lowrank_back, dict(gb=P[8]), ALIAS), (lowrank_back, dict(ga=P[6]), ALIAS),
    (lowrank_back, dict(ws=P[7]), ALIAS), (lowrank_back, dict(ws=P[1]), ALIAS), (lowrank_back, dict(ws=P[5]), ALIAS),
    (balance, dict(dtype=3), ARG), (balance, dict(score=2), ARG), (balance, dict(T=-1), SHAPE),
    (balance, dict(E=0), SHAPE), (balance, dict(E=1025, ld=1025), SHAPE), (balance, dict(k=0), SHAPE),
    (balance, dict(k=17), SHAPE), (balance, dict(ld=15), SHAPE), (balance, dict(S=-1), SHAPE),
    (balance, dict(offsets=None), SHAPE), (balance, dict(S=2 ** 27), SHAPE), (balance, dict(logits=None), NULL),
    (balance, dict(experts=None), NULL), (balance, dict(loss=None), NULL), (balance, dict(counts=None), NULL),
    (balance, dict(logits=P[0] + 2), ARG), (balance, dict(loss=P[3] + 1), ARG), (balance, dict(offsets=P[2] + 2), ARG),
    (balance, dict(loss=P[0]), ALIAS), (balance, dict(counts=P[1]), ALIAS), (balance, dict(counts=P[2]), ALIAS),
    (balance, dict(loss=P[4] + 4), ALIAS), (balance, dict(nbytes=64), ARG), (balance, dict(ws=P[5] + 4), ARG),
    (balance, dict(ws=P[0]), ALIAS), (balance, dict(ws=P[4]), ALIAS),
    (balance_back, dict(dtype=3), ARG), (balance_back, dict(score=-1), ARG), (balance_back, dict(renorm=2), ARG),
    (balance_back, dict(scale=float("inf")), ARG), (balance_back, dict(E=0), SHAPE), (balance_back, dict(ld=3), SHAPE),
    (balance_back, dict(offsets=None), SHAPE), (balance_back, dict(gl=None), NULL), (balance_back, dict(logits=None), NULL),
    (balance_back, dict(counts=None), NULL), (balance_back, dict(experts=None), NULL), (balance_back, dict(out=None), NULL),
    (balance_back, dict(out=P[6] + 2), ARG), (balance_back, dict(gw=P[5] + 2), ARG), (balance_back, dict(out=P[1]), ALIAS),
    (balance_back, dict(out=P[3]), ALIAS), (balance_back, dict(out=P[5]), ALIAS), (balance_back, dict(out=P[0]), ALIAS),
]


@pytest.mark.parametrize("call,args,want", BAD, ids=lambda v: getattr(v, "__name__", None) or str(v))
def test_refused(call, args, want):
    assert call(**args) == want


def test_empty_calls_do_nothing():
    assert lowrank(T=0) == 0 and lowrank(N=0) == 0 and lowrank_back(gx=None, ga=None, gb=None) == 0
    assert balance(S=0) == 0 and balance_back(T=0) == 0
    assert binding.last_kernel() == "none"


def test_sizes():
    assert binding.lowrank_linear_backward_workspace_bytes(0, 8) == 0
    assert binding.lowrank_linear_backward_workspace_bytes(5, 129) == 0
    assert binding.lowrank_linear_backward_workspace_bytes(2 ** 27 + 1, 8) == 0
    assert binding.lowrank_linear_backward_workspace_bytes(100, 8) > 0


def test_without_a_gpu_calls_fail_loudly():
    calls = [("lowrank_linear", [P[0], 0, 64, P[1], P[2], None, P[4], None, P[6], 9, 3, 8, 64, 32, None, 0, None]),
             ("lowrank_linear", [P[0], 0, 64, P[1], P[2], P[3], P[4], P[6], P[6], 900, 3, 8, 64, 32, P[7], 1 << 20, None]),
             ("lowrank_linear_backward", [P[0], P[1], P[2], P[3], 0, P[4], P[5], P[7], P[7], P[8], P[9], 9, 3, 8, 64, 32,
                                          P[10], 1 << 20, None]),
             ("moe_balance", [P[0], 0, 9, 16, 16, P[1], 2, 0, None, 1, P[3], P[4], None, 0, None]),
             ("moe_balance_backward", [P[0], P[1], 0, 9, 16, 16, None, 2, 0, P[3], None, 1, None, 1, 1.0, P[6], None])]
    assert without_gpu(calls) == [binding.IMC_ERR_DEVICE] * len(calls)


def test_torch_level_checks():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):  # not on the GPU
        binding.adapters_linear(x, x, x, None)
    with pytest.raises(TypeError):
        binding.adapters_linear([1.0], x, x, None)
    with pytest.raises(ValueError):
        binding.adapters_linear_backward(x, x, x, x, None)
    with pytest.raises(ValueError):
        binding.balance_loss(x, x.int())
    with pytest.raises(TypeError):
        binding.balance_loss([0.0], x)
    with pytest.raises(ValueError):
        binding.balance_loss_backward(x, x, x.int(), x)


def test_python_module_calls_the_same_entry_points():
    binding._setup()
    for name in ("lowrank_linear", "lowrank_linear_backward", "moe_balance", "moe_balance_backward"):
        zeros = [0.0 if t is binding._dbl else 0 for t in binding.SIGNATURES[name][1]]
        assert getattr(binding._calls, name)(*zeros) == getattr(binding.load(), name)(*zeros) == \
            getattr(binding, name)(*zeros), name
        with pytest.raises(TypeError, match=name):
            getattr(binding._calls, name)(*zeros[1:])
    assert binding._calls.lowrank_linear(P[0], 0, 64, P[1], P[2], P[3], P[4], P[5], P[1], 9, 3, 8, 64, 32, None, 0, None) == ALIAS
    assert binding._calls.moe_balance(P[0], 0, 9, 16, 16, P[1], 2, 0, None, 1, P[0], P[4], None, 0, None) == ALIAS
