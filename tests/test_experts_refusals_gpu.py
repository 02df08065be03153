"""What the expert products refuse on the GPU: with an ArError, and before anything is written."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from allreduce_reduction_emulated_gb300 import _build

    _build.build()


def refused(call, status, text=""):
    from allreduce_reduction_emulated_gb300 import ArError

    with pytest.raises(ArError) as e:
        call()
    assert e.value.status == status and text in str(e.value), str(e.value)


def bf(*shape, value=1.0):
    return torch.full(shape, value, dtype=torch.bfloat16, device="cuda")


def offsets(*values):
    return torch.tensor(values, device="cuda")


@pytest.mark.parametrize("shift", [0, 1])
def test_sizes_beyond_the_limits(shift):
    """Sums long enough to be asked about parts, operands laid out anew: no size of theirs is asked for."""
    from allreduce_reduction_emulated_gb300 import AR_ERR_UNSUPPORTED, experts

    K = (1 << 24) + 8
    x = bf(K + shift)[shift:].view(1, K)
    w = bf(1, 1, K)
    refused(lambda: experts.expert_product(x, w, offsets(0, 1), dtype=torch.float32), AR_ERR_UNSUPPORTED)
    refused(lambda: experts.expert_product(x, w, offsets(0, 1)), AR_ERR_UNSUPPORTED)
    E = 1025
    x, w, off = bf(3, 1024 + shift)[:, shift:], bf(E, 8, 1024), torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    refused(lambda: experts.expert_product(x, w, off), AR_ERR_UNSUPPORTED)
    dy = bf(3, 8)
    refused(lambda: experts.expert_gradients(dy, x, w, off), AR_ERR_UNSUPPORTED)
    refused(lambda: experts.expert_gradients(dy, x, w, off, need_dx=False), AR_ERR_UNSUPPORTED)
