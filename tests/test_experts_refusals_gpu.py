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


def test_a_refused_dw_leaves_dx_alone():
    """dw in the memory of x or dy: nothing is launched, not dx either."""
    from allreduce_reduction_emulated_gb300 import AR_ERR_INVALID_ARG, experts

    rows, N, K = 40, 64, 64
    w, off = bf(1, N, K), offsets(0, rows)
    flat = bf(2 * N * K)
    near, far = flat[:rows * K].view(rows, K), bf(rows, K)
    dx = bf(rows, K, value=7.0)
    for dy, x in ((near, far), (far, near)):
        for dw in (flat[:N * K].view(1, N, K), flat[rows * K - 8:][:N * K].view(1, N, K)):
            refused(lambda: experts.expert_gradients(dy, x, w, off, dx=dx, dw=dw), AR_ERR_INVALID_ARG, "share memory")
            refused(lambda: experts.expert_gradients(dy, x, w, off, dw=dw, need_dx=False), AR_ERR_INVALID_ARG)
    torch.cuda.synchronize()
    assert bool((dx == 7.0).all()) and bool((flat == 1.0).all())
    # right behind x
    dw = flat[rows * K:][:N * K].view(1, N, K)
    assert experts.expert_gradients(far, near, w, off, dx=dx, dw=dw)[1] is dw
    assert bool((dw == float(rows)).all()) and bool((dx == float(N)).all())


def test_long_sums_in_their_inputs():
    """Results that go by way of 32-bit ones are refused in their inputs' memory like any others."""
    from allreduce_reduction_emulated_gb300 import AR_ERR_INVALID_ARG, experts

    N, K = (1 << 18) + 64, 8
    dy, x, w, off = bf(2, N), bf(2, K), bf(1, N, K), offsets(0, 2)
    inside = dy.view(-1)[:2 * K].view(2, K)
    refused(lambda: experts.expert_gradients(dy, x, w, off, dx=inside), AR_ERR_INVALID_ARG, "memory")
    refused(lambda: experts.expert_gradients(dy, x, w, off, dx=inside, need_dw=False), AR_ERR_INVALID_ARG, "memory")
    refused(lambda: experts.expert_product(dy, w.transpose(1, 2), off, out=inside), AR_ERR_INVALID_ARG, "memory")
    inside = w.view(-1)[:2 * K].view(2, K)
    refused(lambda: experts.expert_gradients(dy, x, w, off, dx=inside), AR_ERR_INVALID_ARG, "memory")
    torch.cuda.synchronize()
    assert bool((dy == 1.0).all()) and bool((w == 1.0).all())
    dx, dw = experts.expert_gradients(dy, x, w, off, dx=bf(2, K))
    assert bool((dx == 2.0 ** 18).all()) and bool((dw == 2.0).all())     # 2^18 + 64 rounds to 2^18
