"""Precision of the global norm where every rounding goes the same way: long sums of
equal squares (random data lets the roundings cancel).

Bound: a thread adds at most 16 squares into each of four fp32 accumulators before
these are carried into a compensated sum, so each addition's 2^-24 is of a sum of at most
16 squares: at most 8.5 2^-24 of it; joining the four and the compensated sum's
end 3 2^-24; the block's tree 5 + 8 additions; the partial sums' at most 3 + 5 + 8
(one launch).  40.5 2^-24 = 2.4e-6 of the sum, half of it of the norm, and the root's own
2^-24: 1.3e-6."""
import math

import pytest
import torch

from allreduce_reduction_emulated_gb300.clipping import GradClipper

pytestmark = pytest.mark.gpu
TOL = 1.3e-6


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype,n", [(torch.float32, 40_000_003), (torch.float32, 1_200_000_001),
                                     (torch.bfloat16, 600_000_007), (torch.bfloat16, 1 << 32)],
                         ids=["f32-160MB", "f32-4.8GB", "bf16-1.2GB", "bf16-8.6GB"])
def test_equal_squares(dev, dtype, n):
    g = torch.empty(n, dtype=dtype, device=dev)
    clipper = GradClipper([g])
    for value in (0.010973775, 0.0058268597, 0.022141213, 0.0019666532, 0.9011173, 0.1, 3e-4, 0.75):
        g.fill_(value)
        c = float(g[0])
        want = abs(c) * math.sqrt(n)
        norm = clipper.norm()
        assert abs(float(norm) - want) <= TOL * want, (value, float(norm) / want - 1)
        got = clipper.clip(want / 4, eps=0.0)         # two bits off: the clipped values show the coefficient
        assert torch.equal(got, norm)
        if dtype == torch.float32:
            assert abs(float(g[n // 2]) - c / 4) <= (TOL + 2.0 ** -23) * c / 4


def test_many_launches(dev):
    """More tensors than a launch takes: more partial sums, at most 32 more additions of them."""
    n, count = 300_000, 2000
    flat = torch.full((n * count,), 0.010973775, device=dev)
    clipper = GradClipper(flat.split(n))
    want = float(flat[0]) * math.sqrt(n * count)
    assert abs(float(clipper.norm()) - want) <= (TOL + 16 * 2.0 ** -24) * want


def test_infinite_and_nan_sums(dev):
    """Squares and sums beyond fp32's range make the norm infinite, NaN stays NaN, also behind them."""
    n = 50_000_000
    for where in (0, n // 2, n - 1):
        g = torch.full((n,), 0.01, device=dev)
        g[where] = 2e19
        assert float(GradClipper([g]).norm()) == math.inf
        g[where] = math.inf
        assert float(GradClipper([g]).norm()) == math.inf
        g[(where + 12345) % n] = math.nan
        assert math.isnan(float(GradClipper([g]).norm()))
    g = torch.full((n,), 1.5e16, device=dev)          # every square is finite, their sum is not
    assert float(GradClipper([g]).norm()) == math.inf
