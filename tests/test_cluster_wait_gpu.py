"""A block of a cluster whose bounded wait for the others runs out: the call ends, its rows
are NaN everywhere, no others are, and the next call is not touched.  (The wait is given up
at once here, in a process of its own; nothing is lost on the way.)"""
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
from allreduce_reduction_emulated_gb300 import losses
late = {late}
for T, V, dtype, clusters in ((37, 9001, torch.float32, True), (700, 9001, torch.float32, True),
                              (37, 50003, torch.bfloat16, True), (700, 50003, torch.bfloat16, True),
                              (61, 131072, torch.bfloat16, True), (19, 262000, torch.bfloat16, True),
                              (50, 3001, torch.float32, False)):
    for in_place in (False, True):
        g = torch.Generator(device="cuda").manual_seed(V)
        x = torch.randn(T, V, device="cuda", generator=g).to(dtype)
        y = torch.randint(0, V, (T,), device="cuda", generator=g)
        w = (torch.rand(T, device="cuda", generator=g) < 0.8).float()
        w[0] = 1.0
        adv = torch.randn(T, device="cuda", generator=g)
        lp = torch.log_softmax(x.float(), 1).gather(1, y[:, None]).squeeze(1)
        room = torch.full((T * V + 64,), 7.0, device="cuda", dtype=dtype)
        grad = x if in_place else room[32:32 + T * V].view(T, V)
        r = losses.policy_loss(x, y, lp, adv, weights=w, grad=grad)
        torch.cuda.synchronize()
        assert bool((room[:32] == 7).all()) and bool((room[-32:] == 7).all())
        on = w != 0
        assert not bool(r.grad[~on].any()) and not bool(r.logprobs[~on].any())
        # does a cluster of this shape have such a block?
        hit = bool(torch.isnan(r.loss))
        assert hit == (clusters and late < {{9001: 2, 50003: 4, 131072: 4, 262000: 8, 3001: 1}}[V]), (V, hit)
        nan = torch.isnan(r.grad[on])
        if hit:
            assert bool(nan.all()) and bool(torch.isnan(r.logprobs[on]).all()) and bool(torch.isnan(r.stats).all())
        else:
            assert not bool(nan.any()) and float((r.logprobs - lp)[on].abs().max()) < 1e-4
print("done")
"""


@pytest.mark.parametrize("late", [0, 1, 3, 7])
def test_a_wait_that_runs_out(late):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE.format(root=root, late=late)], capture_output=True, text=True,
                       timeout=300, env={**os.environ, "AR_LATE_BLOCK": str(late)})
    assert r.returncode == 0 and "done" in r.stdout, r.stdout + r.stderr
