"""A stream of another device is refused before anything is launched there."""
import pytest
import torch

from allreduce_reduction_emulated_gb300 import _build, experts, losses
from test_train_abi import OnGpu, refused


class OfAnother:
    device_index, cuda_stream = 1, 0


@pytest.fixture(autouse=True)
def first(monkeypatch):
    _build.build()
    for m in (losses, experts):
        monkeypatch.setattr(m, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: pytest.fail("entered"))


def bf(*shape):
    return OnGpu.of(torch.zeros(shape, dtype=torch.bfloat16))


def test_experts():
    x, dy, w, off = bf(6, 8), bf(6, 16), bf(3, 16, 8), OnGpu.of(torch.tensor([0, 2, 4, 6]))
    refused(lambda: experts.expert_product(x, w, off, stream=OfAnother()), "it is on cuda:1")
    refused(lambda: experts.expert_gradients(dy, x, w, off, stream=OfAnother()), "it is on cuda:1")


def test_losses():
    x, y, v = bf(4, 8), OnGpu.of(torch.zeros(4, dtype=torch.int64)), OnGpu.of(torch.zeros(4))
    refused(lambda: losses.token_logprobs(x, y, stream=OfAnother()), "it is on cuda:1")
    refused(lambda: losses.policy_loss(x, y, v, v, stream=OfAnother()), "it is on cuda:1")
