"""Adapters whose weights are copied by 8 or 4 bytes, with the layout anywhere in memory.

Ranks and widths that are multiples of 4 or 2 but not of 8: every other piece of a unit is past
the end and reads nothing.  The layout begins at an 8-byte boundary and at none.
"""
import pytest
import torch

from addmm_implicit_im2col_gb300 import binding
from test_gpu_adapters import TYPES, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("place", [0, 1])
@pytest.mark.parametrize("r", [4, 12, 20, 6, 2, 36])
@pytest.mark.parametrize("K,N,which", [(120, 264, "mixed"), (124, 132, "runs"), (130, 66, "mixed")])
def test_pieces_past_the_end(K, N, which, r, place, dtype):
    T, L = 9000 // r + 1200, 3
    c = Case(r + place, T, L, r, K, N, dtype, which=which)
    data = torch.full((c.layout.data.numel() + 3,), -1, dtype=torch.int32, device="cuda")
    assert data.data_ptr() % 16 == 0
    data[place:place + c.layout.data.numel()] = c.layout.data
    c.layout = binding.ExpertsLayout(data[place:], T, 1, L)
    assert c.layout.data.data_ptr() % 8 == 4 * place
    c.check()
