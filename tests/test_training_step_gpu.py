"""The operators together, as the example runs them: loss, gradients, bucket
all-reduces, clipping and update on emulated ranks, against 64-bit autograd."""
import os
import sys

import pytest
import torch

import allreduce_reduction_emulated_gb300 as ar
from allreduce_reduction_emulated_gb300 import losses

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)
    import training_step

    return training_step


@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_trains(example, kind):
    """On one batch the loss falls, and every step's norm is finite and positive."""
    history = example.run(kind, steps=25)
    assert all(norm > 0 and norm < 1e4 for _, norm in history)
    assert history[-1][0] < history[0][0] - 0.01


@pytest.mark.parametrize("max_norm", [1e-3, 1e3])
def test_one_step_against_autograd(example, max_norm):
    """Weights after one step = weights - rate * clipped mean gradient of the ranks'
    losses in 64 bits.  The GEMMs run in fp32 (no TF32 here) over at most 1000
    terms: 1e-4 of the update's size covers them."""
    torch.backends.cuda.matmul.allow_tf32 = False
    ranks, features, hidden, vocab = 3, 20, 30, 501
    step = example.Step(ranks, features, hidden, vocab, max_norm=max_norm, bucket=4000)
    try:
        xs, args = example.preference_batch(step, 3, 9, features, vocab)
        w1, w2 = (w.double().clone().requires_grad_() for w in (step.w1, step.w2))
        total = 0.0
        for x, (y, off, ref) in zip(xs, args):
            logp = torch.log_softmax(torch.tanh(x.double() @ w1) @ w2, 1).gather(1, y[:, None]).squeeze(1)
            gain = [(logp[a:b] - ref[a:b].double() * 1.01).sum() for a, b in zip(off.tolist(), off.tolist()[1:])]
            z = 0.5 * torch.stack([a - b for a, b in zip(gain[0::2], gain[1::2])])
            total = total - torch.nn.functional.logsigmoid(z).mean() / ranks
        g1, g2 = torch.autograd.grad(total, (w1, w2))
        norm = float((g1.square().sum() + g2.square().sum()).sqrt())
        coef = min(1.0, max_norm / (norm + 1e-6))
        want = [(w - step.rate * coef * g).detach() for w, g in ((w1, g1), (w2, g2))]

        def loss(r, logits):
            y, off, ref = args[r]
            return losses.preference_loss(logits, y, off, ref * 1.01, beta=0.5, grad=logits)

        each, got = step(xs, loss)
        assert ar.ar_get_status(step.comm) == ar.AR_SUCCESS
        assert abs(float(got) - norm) <= 1e-4 * norm
        assert abs(float(each.mean()) - float(total.detach())) <= 1e-5 * abs(float(total.detach()))
        for w, v, g in ((step.w1, want[0], g1), (step.w2, want[1], g2)):
            assert float((w.double() - v).abs().max()) <= 1e-4 * step.rate * coef * float(g.abs().max()) + 3e-7
        for r in range(1, ranks):                     # the reduced gradients, before clipping, on the other ranks
            assert torch.equal(step.grads[r], step.grads[1])
    finally:
        step.close()
