"""Numbers of adapters whose table fills up the shared memory behind the second product's rings.

The table takes 8 bytes an adapter, the rings what is left in steps of some KB: every number of
adapters has to find room, however little is left over.
"""
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding
from test_gpu_adapters import TYPES, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("r", [16, 24, 40, 64, 72, 128])
@pytest.mark.parametrize("L", [125, 126, 127, 136, 148, 165, 166, 260, 290])
@pytest.mark.parametrize("K,N", [(40, 132), (24, 56), (33, 71)])
def test_every_number_of_adapters(L, r, K, N, dtype):
    Case(L + r, 20 * L, L, r, K, N, dtype, which="runs").check()


def test_every_number_of_adapters_has_room():
    """Every number up to the most, small calls: none is refused."""
    for dtype in TYPES:
        x = torch.zeros(1, 8, dtype=dtype, device="cuda")
        for L in list(range(1, 1025, 7)) + list(range(120, 170)) + [1023, 1024]:
            for r in (1, 20, 33, 65, 97, 113):
                a, b = torch.zeros(L, r, 8, dtype=dtype, device="cuda"), torch.zeros(L, 5, r, dtype=dtype, device="cuda")
                layout = binding.experts_layout(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), L)
                grads = binding.adapters_linear_backward(x[:, :5].contiguous(), x, a, b, layout)
                assert not any(g.any() for g in grads)
