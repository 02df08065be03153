"""policy_loss where its terms are far apart in size: terms of weight 0, near-certain tokens,
very long rows, many rows."""
import math

import pytest
import torch

import train_util as tu
from allreduce_reduction_emulated_gb300 import losses

pytestmark = pytest.mark.gpu
INF = math.inf
BOTH = [torch.float32, torch.bfloat16]
IDS = ["f32", "bf16"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.mark.parametrize("V", [300, 40000, 600001])
def test_kl_term_of_coefficient_zero_is_left_out(dev, V):
    """A reference given for the statistic alone: where e^d is infinite the statistic is, not the loss."""
    g = torch.Generator(device=dev).manual_seed(V)
    T = 6
    logits = torch.randn(T, V, device=dev, generator=g)
    y = torch.arange(T, device=dev)
    logits[2, 2] = -200.0
    old = losses.token_logprobs(logits, y) - 0.1
    adv = torch.randn(T, device=dev, generator=g)
    ref = old.clone()
    ref[2] = 0.0
    plain = losses.policy_loss(logits, y, old, adv)
    r = losses.policy_loss(logits, y, old, adv, ref_logprobs=ref, kl_coef=0.0)
    assert torch.equal(r.loss, plain.loss) and torch.equal(r.grad, plain.grad)
    assert float(r.kl) == INF and math.isfinite(float(r.loss))
