"""A data-parallel step of an expert layer on P emulated ranks of one GPU, all of its products but the
head's in this library:

  each rank   rows sorted by the expert that the router chose -> expert products -> tanh -> logits ->
              policy loss and the gradient of the logits -> gradients of the head and of the experts'
              weights (32 bits, straight into the rank's flat buffer);
  all ranks   bucket all-reduces (ring, mean), the global norm and clipping, the orthogonalised update with
              momentum, new weights.

    python examples/expert_step.py [--steps 20] [--ranks 2] [--experts 4]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import allreduce_reduction_emulated_gb300 as ar
from allreduce_reduction_emulated_gb300 import experts, losses
from allreduce_reduction_emulated_gb300.buckets import BucketReducer
from allreduce_reduction_emulated_gb300.clipping import GradClipper
from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer


class ExpertStep:
    """Weights (32-bit masters, 16-bit copies), one flat gradient buffer per rank, and the handles kept across steps."""

    def __init__(self, ranks: int, features: int, hidden: int, vocab: int, count: int, max_norm: float = 1.0,
                 rate: float = 0.02, seed: int = 0, bucket: int = 1 << 16):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        shapes = [(hidden, vocab), (count, hidden, features)]        # backward order: the head's gradients first
        self.head = torch.randn(shapes[0], device="cuda", generator=gen) / hidden ** 0.5
        self.experts = torch.randn(shapes[1], device="cuda", generator=gen) / features ** 0.5
        self.ranks, self.rate, self.max_norm = ranks, rate, max_norm
        sizes = [self.head.numel(), self.experts.numel()]
        self.flat = [torch.zeros(sum(sizes), device="cuda") for _ in range(ranks)]
        self.grads = [[part.view(s) for part, s in zip(f.split(sizes), shapes)] for f in self.flat]
        self.comm = ar.ar_init(ranks)
        self.reducer = BucketReducer(self.comm, self.flat, bucket, scale=1.0 / ranks)
        # the reduced gradients are the same on every rank; rank 0's are clipped and used
        self.clipper = GradClipper(self.grads[0])
        self.momentum = [torch.zeros(s, device="cuda") for s in shapes]
        self.ortho = Orthogonalizer(self.grads[0], momentum=self.momentum, scale="shape")

    def close(self):
        ar.ar_destroy(self.comm)

    def __call__(self, batches):
        """batches[r]: rank r's rows (bf16, sorted by expert), offsets, tokens, old log-probabilities, advantages.
        Returns (losses, norm), on the GPU."""
        weights = self.experts.to(torch.bfloat16)
        self.reducer.reset()
        done = []
        for r, (x, offsets, y, old, advantages) in enumerate(batches):
            h = torch.tanh(experts.expert_product(x, weights, offsets, dtype=torch.float32))
            logits = h @ self.head
            result = losses.policy_loss(logits, y, old, advantages, grad=logits)
            done.append(result.loss)
            torch.mm(h.t(), result.grad, out=self.grads[r][0])
            dh = ((result.grad @ self.head.t()) * (1 - h * h)).to(torch.bfloat16)
            experts.expert_gradients(dh, x, weights, offsets, dw=self.grads[r][1], need_dx=False)
        ready = torch.cuda.Event()
        ready.record()
        self.reducer.ready(self.flat[0].numel(), ready)
        torch.cuda.current_stream().wait_event(self.reducer.finish())
        norm = self.clipper.clip(self.max_norm)
        for w, u in zip((self.head, self.experts), self.ortho.update()):
            w.sub_(u, alpha=self.rate)
        return torch.stack(done), norm


def batch(step: ExpertStep, rows: int, features: int, vocab: int, count: int, seed: int = 1):
    """Each rank's rows as a router leaves them: sorted by expert, an uneven number for each, the last few for none."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    batches = []
    for _ in range(step.ranks):
        x = torch.randn(rows, features, device="cuda", generator=gen).to(torch.bfloat16)
        chosen = torch.randint(0, count * count, (rows - 3,), device="cuda", generator=gen).float().sqrt().long().sort()[0]
        offsets = torch.cat([chosen.new_zeros(1), torch.bincount(chosen, minlength=count).cumsum(0)])
        y = torch.randint(0, vocab, (rows,), device="cuda", generator=gen)
        advantages = torch.randn(rows, device="cuda", generator=gen)
        h = torch.tanh(experts.expert_product(x, step.experts.to(torch.bfloat16), offsets, dtype=torch.float32))
        batches.append((x, offsets, y, losses.token_logprobs(h @ step.head, y), advantages))
    return batches


def run(steps: int = 20, ranks: int = 2, features: int = 64, hidden: int = 96, vocab: int = 1000, count: int = 4):
    """Trains on one batch; returns [(mean loss over the ranks, gradient norm), ...]."""
    step = ExpertStep(ranks, features, hidden, vocab, count)
    try:
        batches = batch(step, 200, features, vocab, count)
        history = [step(batches) for _ in range(steps)]
        status = ar.ar_get_status(step.comm)           # waits for the GPU
        if status != ar.AR_SUCCESS:
            raise RuntimeError(ar.ar_get_error_string(status))
        return [(float(ls.mean()), float(norm)) for ls, norm in history]
    finally:
        step.close()


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--ranks", type=int, default=2)
    p.add_argument("--experts", type=int, default=4)
    a = p.parse_args()
    for i, (loss, norm) in enumerate(run(a.steps, a.ranks, count=a.experts)):
        print(f"step {i:3d}  loss {loss:+.5f}  gradient norm {norm:.4f}")


if __name__ == "__main__":
    main()
