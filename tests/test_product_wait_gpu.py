"""A block of the products that gives up: the call ends, what the block has not computed is NaN, everything
else is right or NaN, nothing beside the results is written, and the next call is not touched.
(It gives up at once here, in a process of its own; the blocks that wait for it run into their own limits.)"""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

CODE = """
import sys
import torch
sys.path.insert(0, {root!r})
from allreduce_reduction_emulated_gb300 import experts
from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

def normal(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=g)

def check(got, want, tol, some):
    torch.cuda.synchronize()
    nan = torch.isnan(got)
    assert some is None or bool(nan.any()) == some, (some, int(nan.sum()), got.shape)
    off = torch.where(nan, 0.0, (got.double() - want).abs())
    assert float(off.max()) <= tol, float(off.max())

for rows, K, N in ((700, 200, 300), (3000, 512, 4096)):      # blocks alone, pairs of blocks
    counts = [rows // 3, rows // 2]
    off = torch.tensor([0, counts[0], sum(counts)], device="cuda")
    x, w, dy = normal(rows, K).bfloat16(), normal(2, N, K, seed=1).bfloat16(), normal(rows, N, seed=2).bfloat16()
    room = torch.full((rows * N + 128,), 7.0, device="cuda", dtype=torch.bfloat16)
    y = room[64:-64].view(rows, N)
    experts.expert_product(x, w, off, out=y)
    a, b = counts[0], sum(counts)
    want = torch.cat([x[:a].double() @ w[0].double().t(), x[a:b].double() @ w[1].double().t()])
    check(y[:b], want, float(want.abs().max()) / 200, True)
    assert bool((room[:64] == 7).all()) and bool((room[-64:] == 7).all()) and bool((y[b:] == 7).all())
    _, dw = experts.expert_gradients(dy, x, w, off, need_dx=False, dw_dtype=torch.float32)
    want = torch.stack([dy[:a].double().t() @ x[:a].double(), dy[a:b].double().t() @ x[a:b].double()])
    check(dw, want, float(want.abs().max()) / 200, True)

for shape in ((200, 330), (20, 512, 700)):
    g = normal(*shape)
    (u,) = Orthogonalizer([g]).update()
    torch.cuda.synchronize()
    assert bool(torch.isnan(u).any())
    if len(shape) == 2:
        assert bool(torch.isnan(u).all())      # every element of a step depends on every block's
(u,) = Orthogonalizer([normal(100, 120)]).update()   # a matrix whole in one block: no block waits for another
torch.cuda.synchronize()
assert not bool(torch.isnan(u).any())
print("done")
"""


@pytest.mark.parametrize("late", [0, 1])
def test_a_block_that_gives_up(late):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE.format(root=root)], capture_output=True, text=True, timeout=300,
                       env={**os.environ, "AR_LATE_BLOCK": str(late)})
    assert r.returncode == 0 and "done" in r.stdout, r.stdout + r.stderr
