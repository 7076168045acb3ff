"""First calls of the same kernels by several host threads at once, of different sizes.

What a kernel may take of shared memory is set at its first call, and the sizes below need
different amounts of it; every process has only one first call, so each run is one of its own.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import threading
import torch
from addmm_implicit_im2col_gb300 import binding

gen = torch.Generator().manual_seed(1)


def normal(*shape, dtype):
    return torch.randn(*shape, generator=gen).to(dtype).cuda()


def balance(dtype, T, E):
    x = normal(T, E, dtype=dtype)
    experts = x.float().topk(2, -1).indices.int().contiguous()
    return lambda: binding.balance_loss(x, experts)


def adapters(dtype, T, L, r, back):
    K, N = 256, 384
    x, a, b = normal(T, K, dtype=dtype), normal(L, r, K, dtype=dtype), normal(L, N, r, dtype=dtype)
    layout = binding.experts_layout(torch.randint(0, L, (T, 1), generator=gen).int().cuda(), L)
    if not back:
        return lambda: (binding.adapters_linear(x, a, b, layout),)
    grad = normal(T, N, dtype=dtype)
    return lambda: binding.adapters_linear_backward(grad, x, a, b, layout)


ranks = (8, 128, 40, 72)
groups = []
for dtype in (torch.float32, torch.bfloat16, torch.float16):
    for sizes in ((1024, 513, 600, 800), (512, 257, 300, 400)):
        groups.append([balance(dtype, 8, E) for E in sizes])
        groups.append([balance(dtype, 700, E) for E in sizes])
    groups.append([adapters(dtype, 40, 5, r, False) for r in ranks])
    groups.append([adapters(dtype, 3000, 2, r, False) for r in ranks])
    groups.append([adapters(dtype, 3000, 2, r, True) for r in ranks])
torch.cuda.synchronize()
wrong = []
for number, calls in enumerate(groups):
    at_once, results = threading.Barrier(len(calls)), [None] * len(calls)

    def one(i):
        at_once.wait()
        try:
            results[i] = calls[i]()
        except Exception as error:
            wrong.append((number, i, "at once", str(error)))

    threads = [threading.Thread(target=one, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i, call in enumerate(calls):
        try:
            alone = call()
        except Exception as error:
            wrong.append((number, i, "alone afterwards", str(error)))
            continue
        if results[i] is not None and not all(torch.equal(p, q) for p, q in zip(results[i], alone)):
            wrong.append((number, i, "other results"))
torch.cuda.synchronize()
assert not wrong, wrong
"""


@pytest.mark.parametrize("run", range(3))
def test_first_calls_at_the_same_time(run):
    done = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
