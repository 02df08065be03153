"""Sums over a million products, all of one sign: what each addition loses would show in their mean."""
import pytest
import torch

from experts_util import product64, weight_gradient64

pytestmark = pytest.mark.gpu

LENGTH = (1 << 20) + 24


@pytest.fixture(scope="module", autouse=True)
def built():
    from allreduce_reduction_emulated_gb300 import _build

    _build.build()


def positive(rows, cols, seed, along):
    """Uniform values; along 0 / 1: every column / row times a factor of 1 to 4, so that sums lie anywhere in a step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    factor = 1 + 3 * torch.rand((1, cols) if along == 0 else (rows, 1), device="cuda", generator=gen)
    return (torch.rand(rows, cols, device="cuda", generator=gen) * factor).bfloat16()


def assert_long(got, want):
    # A run of 960 is off by at most (60 + 16) 2^-23 of itself, each of the 1093 additions of runs by half a unit:
    # 7.5e-5.  Rounding to bf16 is off by at most 2^-8, evenly to both sides: the mean of n by 2^-8 / sqrt(3 n), and by five
    # times that hardly ever.
    lost = 76 * 2.0 ** -23 + 1093 * 2.0 ** -24
    off = (got.double() - want) / want
    assert float(off.abs().max()) <= 2.0 ** -8 * (1 + lost) + lost
    assert float(off.mean().abs()) <= lost + 5 * 2.0 ** -8 / (3 * off.numel()) ** 0.5


@pytest.mark.parametrize("given", [False, True])
def test_long_product(given):
    from allreduce_reduction_emulated_gb300 import experts

    x, w = positive(48, LENGTH, 1, 1), positive(2 * 96, LENGTH, 2, 1).view(2, 96, LENGTH)
    off = torch.tensor([3, 30, 41], device="cuda")
    out = torch.full((48, 96), 7.0, device="cuda", dtype=torch.bfloat16) if given else None
    y = experts.expert_product(x, w, off, out=out)
    assert y.dtype == torch.bfloat16 and (not given or y is out)
    assert_long(y[3:41], product64(x, w, off)[0][3:41])
    rest = torch.cat([y[:3], y[41:]])
    assert torch.equal(rest, torch.full_like(rest, 7.0 if given else 0.0))


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_long_gradients(layout):
    from allreduce_reduction_emulated_gb300 import experts

    dy, x = positive(LENGTH, 72, 3, 0), positive(LENGTH, 104, 4, 0)
    w = torch.zeros((3, 72, 104) if layout == "out_in" else (3, 104, 72), device="cuda", dtype=torch.bfloat16)
    if layout == "in_out":
        w = w.transpose(1, 2)
    off = torch.tensor([0, 40, 40, LENGTH - 3], device="cuda")
    want = weight_gradient64(dy, x, off, 3)[0]
    _, dw = experts.expert_gradients(dy, x, w, off, need_dx=False)
    assert dw.dtype == torch.bfloat16 and dw.stride() == w.stride()
    assert_long(dw[2], want[2])
    assert not dw[1].any()
    # added to what is there, which is rounded with the sum; an expert without rows keeps its own
    before = dw.clone()
    _, more = experts.expert_gradients(dy, x, w, off, dw=dw, accumulate=True, need_dx=False)
    assert more is dw
    assert_long(dw[2], want[2] + before[2].double())
    assert torch.equal(dw[1], before[1])
