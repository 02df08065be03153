"""A single row has no stride of its own, whatever its tensor says: in refusals too."""
import pytest
import torch

from allreduce_reduction_emulated_gb300 import _build, experts, losses
from test_train_abi import OnGpu, refused


@pytest.fixture(autouse=True)
def on_gpu(monkeypatch):
    _build.build()
    for m in (losses, experts):
        monkeypatch.setattr(m, "_current_device", lambda: 0)


@pytest.mark.parametrize("stride", [0, 3, 8, 100])
def test_dx_in_x(stride):
    g = OnGpu.of
    flat = torch.zeros(200, dtype=torch.bfloat16)
    dy, w = g(torch.zeros(1, 16, dtype=torch.bfloat16)), g(torch.zeros(2, 16, 8, dtype=torch.bfloat16))
    x, off = g(flat.as_strided((1, 8), (stride, 1))), g(torch.tensor([0, 1, 1]))
    for at in (0, 3, 7):
        dx = g(flat.as_strided((1, 8), (stride, 1), at))
        refused(lambda: experts.expert_gradients(dy, x, w, off, dx=dx), "dx and x share")
    assert not experts._shared(x, g(flat.as_strided((1, 8), (stride, 1), 8)))
