"""A data-parallel post-training step on P emulated ranks of one GPU, with the
whole of it in this library but the model's matrix products:

  each rank   logits of its own tokens -> policy or preference loss and the
              gradient of the logits -> gradients of the weights, written into the
              rank's flat buffer in backward order;
  all ranks   bucket all-reduces (ring, mean) on a second stream as soon as a
              weight's gradients are written; then the global norm, clipping, update.

    python examples/training_step.py [--loss policy|preference] [--steps 20] [--ranks 4]

The model is a two-layer head over fixed random features: x -> tanh(x W1) W2.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import allreduce_reduction_emulated_gb300 as ar
from allreduce_reduction_emulated_gb300 import losses
from allreduce_reduction_emulated_gb300.buckets import BucketReducer
from allreduce_reduction_emulated_gb300.clipping import GradClipper


class Step:
    """Weights, one flat gradient buffer per rank, and the handles kept across steps."""

    def __init__(self, ranks: int, features: int, hidden: int, vocab: int, max_norm: float = 1.0, rate: float = 0.5,
                 seed: int = 0, bucket: int = 1 << 16):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.w1 = torch.randn(features, hidden, device="cuda", generator=gen) / features ** 0.5
        self.w2 = torch.randn(hidden, vocab, device="cuda", generator=gen) / hidden ** 0.5
        self.ranks, self.rate, self.max_norm = ranks, rate, max_norm
        # backward order: the last layer's gradients first
        self.sizes = [self.w2.numel(), self.w1.numel()]
        self.grads = [torch.zeros(sum(self.sizes), device="cuda") for _ in range(ranks)]
        self.comm = ar.ar_init(ranks)
        self.reducer = BucketReducer(self.comm, self.grads, bucket, scale=1.0 / ranks)
        # the reduced gradients are the same on every rank; rank 0's are clipped and used
        self.clipper = GradClipper(self.grads[0].split(self.sizes))

    def close(self):
        ar.ar_destroy(self.comm)

    def logits(self, x):
        z = torch.tanh(x @ self.w1)
        return z, z @ self.w2

    def __call__(self, xs, loss):
        """One step: xs[r] is rank r's features, loss(r, logits) its PolicyLoss or
        PreferenceLoss with the gradient in place.  Returns (losses, norm), on the GPU."""
        n2 = self.sizes[0]
        compute = torch.cuda.current_stream()
        self.reducer.reset()
        done, hidden = [], []
        for r, x in enumerate(xs):
            z, logits = self.logits(x)
            result = loss(r, logits)
            done.append(result.loss)
            torch.mm(z.t(), result.grad, out=self.grads[r][:n2].view_as(self.w2))
            hidden.append(result.grad @ self.w2.t() * (1 - z * z))
        ready = torch.cuda.Event()
        ready.record(compute)
        self.reducer.ready(n2, ready)                  # W2's buckets, while W1's gradients are computed
        for r, (x, dz) in enumerate(zip(xs, hidden)):
            torch.mm(x.t(), dz, out=self.grads[r][n2:].view_as(self.w1))
        ready = torch.cuda.Event()
        ready.record(compute)
        self.reducer.ready(sum(self.sizes), ready)
        compute.wait_event(self.reducer.finish())
        norm = self.clipper.clip(self.max_norm)
        g2, g1 = self.grads[0].split(self.sizes)
        self.w2.sub_(g2.view_as(self.w2), alpha=self.rate)
        self.w1.sub_(g1.view_as(self.w1), alpha=self.rate)
        return torch.stack(done), norm


def policy_batch(step: Step, tokens: int, features: int, vocab: int, seed: int = 1):
    """Each rank's rollout: features, sampled tokens, advantages, the old policy's log-probabilities."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    xs, args = [], []
    for _ in range(step.ranks):
        x = torch.randn(tokens, features, device="cuda", generator=gen)
        y = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
        adv = torch.randn(tokens, device="cuda", generator=gen)
        old = losses.token_logprobs(step.logits(x)[1], y)
        xs.append(x)
        args.append((y, old, adv))
    return xs, args


def preference_batch(step: Step, pairs: int, longest: int, features: int, vocab: int, seed: int = 1):
    """Each rank's pairs: features and tokens of all answers, offsets, the reference's log-probabilities."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    xs, args = [], []
    for _ in range(step.ranks):
        n = torch.randint(1, longest + 1, (2 * pairs,), device="cuda", generator=gen)
        off = torch.cat([n.new_zeros(1), n.cumsum(0)])
        tokens = int(off[-1])
        x = torch.randn(tokens, features, device="cuda", generator=gen)
        y = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
        ref = losses.token_logprobs(step.logits(x)[1], y)
        xs.append(x)
        args.append((y, off, ref))
    return xs, args


def run(kind: str = "policy", steps: int = 20, ranks: int = 4, features: int = 64, hidden: int = 96, vocab: int = 1000):
    """Trains on one batch; returns [(mean loss over the ranks, gradient norm), ...]."""
    step = Step(ranks, features, hidden, vocab)
    try:
        if kind == "policy":
            xs, args = policy_batch(step, 200, features, vocab)

            def loss(r, logits):
                y, old, adv = args[r]
                return losses.policy_loss(logits, y, old, adv, ref_logprobs=old, kl_coef=0.01, grad=logits)
        else:
            xs, args = preference_batch(step, 8, 24, features, vocab)

            def loss(r, logits):
                y, off, ref = args[r]
                return losses.preference_loss(logits, y, off, ref, beta=0.5, grad=logits)
        history = [step(xs, loss) for _ in range(steps)]
        status = ar.ar_get_status(step.comm)           # waits for the GPU
        if status != ar.AR_SUCCESS:
            raise RuntimeError(ar.ar_get_error_string(status))
        return [(float(ls.mean()), float(norm)) for ls, norm in history]
    finally:
        step.close()


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--loss", choices=("policy", "preference"), default="policy")
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--ranks", type=int, default=4)
    a = p.parse_args()
    for i, (loss, norm) in enumerate(run(a.loss, a.steps, a.ranks)):
        print(f"step {i:3d}  loss {loss:+.5f}  gradient norm {norm:.4f}")


if __name__ == "__main__":
    main()
