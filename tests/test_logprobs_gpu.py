"""token_logprobs of near-certain tokens in every shape: wherever in its row the one large
logit stands, what came before it in its thread's sum stays."""
import math

import pytest
import torch

from allreduce_reduction_emulated_gb300 import losses

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(3000, 9001), (2600, 30000), (7, 9001), (5, 131072), (200, 100003), (3, 1 << 20)])
def test_near_certain_tokens(dev, T, V, dtype):
    """The large logit at the row's start, middle and end: lp = -log(1 + rest) with a rest of 4e-7 and below.  A
    thread adds its own next three logits or slots to the maximum's 1 and may lose them, 32 of V terms; 1% of
    the rest covers that and what e^z rounds (2^-22 + 24 2^-23)."""
    g = torch.Generator(device=dev).manual_seed(V)
    logits = (-24.0 + torch.rand(T, V, device=dev, generator=g)).to(dtype)
    x = logits.double().exp().sum(1)
    rows = torch.arange(T, device=dev)
    y = torch.where(rows % 3 == 0, rows % 50, torch.where(rows % 3 == 1, V // 2 + rows % 50, V - 1 - rows % 50))
    rest = x - logits.double()[rows, y].exp()
    logits[rows, y] = 0.0
    want = -torch.log1p(rest)
    lp = losses.token_logprobs(logits, y)
    off = (lp.double() - want).abs() / want.abs()
    assert float(off.max()) <= 0.01, [float(off[rows % 3 == k].max()) for k in range(3) if k < T]
    assert math.isfinite(float(lp.sum()))
