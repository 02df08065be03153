"""The products of expert layers, their gradients and the orthogonalised update together, as the example runs
them with the loss, the all-reduce and clipping: one step against 64-bit autograd."""
import os
import sys

import pytest
import torch

from orthogonal_util import update64

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)
    import expert_step

    return expert_step


def test_runs(example):
    history = example.run(steps=3)
    assert len(history) == 3 and all(norm > 0 and norm < 1e4 and loss == loss for loss, norm in history)


@pytest.mark.parametrize("count,features,hidden,vocab", [(3, 40, 56, 301), (2, 72, 200, 150)])
def test_gradients_and_updates_against_autograd(example, count, features, hidden, vocab):
    torch.backends.cuda.matmul.allow_tf32 = False
    step = example.ExpertStep(2, features, hidden, vocab, count, max_norm=1e6, bucket=4000)
    try:
        batches = example.batch(step, 150, features, vocab, count)
        head = step.head.double().clone().requires_grad_()
        w = step.experts.to(torch.bfloat16).double().requires_grad_()     # what the products see
        total = 0.0
        for x, off, y, old, adv in batches:
            off = off.tolist()
            z = torch.cat([x[a:b].double() @ w[e].t() for e, (a, b) in enumerate(zip(off, off[1:]))]
                          + [torch.zeros(len(x) - off[-1], hidden, dtype=torch.float64, device="cuda")])
            lp = torch.log_softmax(torch.tanh(z) @ head, 1).gather(1, y[:, None]).squeeze(1)
            r = (lp - old.double()).exp()
            total = total - torch.minimum(r * adv, r.clamp(0.8, 1.2) * adv).mean() / 2
        want = torch.autograd.grad(total, (head, w))
        before = [step.head.clone(), step.experts.clone()]
        step(batches)
        torch.cuda.synchronize()
        # The head's gradient is fp32 throughout: 1e-4 of its 2-norm.  The experts' goes through dh in bf16, each
        # element off by half a step, 2^-8 / sqrt(3) of its value in random directions: 2.3e-3.
        for g, t, tol in zip(step.grads[0], want, (1e-4, 2.3e-3 + 1e-4)):
            assert float((g.double() - t).norm()) <= tol * float(t.norm())
        # And the update is made of the gradients that are there: 5e-3 of its 2-norm, and w - rate u in fp32.  An
        # expert with fewer rows than features has a gradient of less than full rank; in the directions that it lacks
        # fp16 puts 2.8e-4 of X's 2-norm (1 of the first X, at most 1.2 of the later ones) per matrix, which grows by
        # 3.4445 a step: 2.8e-4 (485 + 1.2 (141 + 41 + 12 + 3.4 + 1)) = 0.2.
        lacking = [0.0, 0.2 * count ** 0.5]
        for g, w0, w1, more in zip(step.grads[0], before, (step.head, step.experts), lacking):
            m, n = g.shape[-2:]
            u, _ = update64(g, torch.zeros_like(g), scale=max(1.0, m / n) ** 0.5)
            got = (w0.double() - w1.double()) / step.rate
            rounding = 2.0 ** -24 * float(w0.norm()) / step.rate
            assert float((got - u).norm()) <= 5e-3 * float(u.norm()) + rounding + more
    finally:
        step.close()
