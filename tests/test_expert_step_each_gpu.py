"""The orthogonalised update of each expert by itself, as the example makes it: full rank to what fp16 leaves of its own
singular values, less than that with what fp16 puts into the directions that it lacks."""
import os
import sys

import pytest
import torch

from orthogonal_util import update64

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("count,features,hidden,vocab", [(3, 40, 56, 301), (2, 72, 200, 150)])
def test_update_of_each_expert(count, features, hidden, vocab):
    import __graft_entry__

    __graft_entry__.build()
    import expert_step

    step = expert_step.ExpertStep(2, features, hidden, vocab, count, max_norm=1e6, bucket=4000)
    try:
        batches = expert_step.batch(step, 150, features, vocab, count)
        rows = sum(off.diff() for _, off, *_ in batches).tolist()
        before = step.experts.clone()
        step(batches)
        torch.cuda.synchronize()
        got = (before.double() - step.experts.double()) / step.rate
        least, full = min(hidden, features), 0
        for e in range(count):
            g = step.grads[0][1][e]
            u = update64(g, torch.zeros_like(g), scale=max(1.0, hidden / features) ** 0.5)[0]
            # fp16 puts 2.8e-4 of X's 2-norm, 1, into `least` directions evenly, which is relative to each direction's
            # singular value s from then on; later steps add as much at most, as s has grown (sqrt(2)).  bf16's half
            # step is 2.3e-3, and w - rate u is rounded to fp32.
            s = torch.linalg.svdvals(g.double() / g.double().norm())
            tol = 2.3e-3 + 2 ** 0.5 * 2.8e-4 * float((1 / (s * s * least)).mean().sqrt())
            more = 2.0 ** -24 * float(before[e].norm()) / step.rate
            if rows[e] < least:  # 2.8e-4 in each step's X, 1 of the first and 1.2 of the later ones, times 3.4445 a step
                tol, more = 5e-3, more + 0.2
            else:
                full += 1
                assert tol < 2e-2, "a full rank that says little"
            off = float((got[e] - u).norm())
            assert off <= tol * float(u.norm()) + more, (e, rows[e], off / float(u.norm()), tol)
        assert full
    finally:
        step.close()
