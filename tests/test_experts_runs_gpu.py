"""32-bit results of sums in several runs of 960 products, whole ones and of last slices, in pairs of blocks and alone."""
import pytest
import torch

from experts_util import assert_sum, product64, weight_gradient64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from allreduce_reduction_emulated_gb300 import _build

    _build.build()


def normal(shape, seed, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=gen).to(dtype)


@pytest.mark.parametrize("counts,N,K", [([1300, 0, 1000, 700], 1500, 2500),     # pairs
                                        ([300, 40, 129, 1], 1030, 1921),        # blocks alone
                                        ([1921, 961, 960, 2000], 1100, 1300)])
def test_runs(counts, N, K):
    from allreduce_reduction_emulated_gb300 import experts, library

    E, rows = len(counts), sum(counts) + 2
    off = torch.tensor([0] + counts).cumsum(0).cuda()
    x, dy, w = normal((rows, K), 1), normal((rows, N), 2), normal((E, N, K), 3)
    x[-2:], dy[-2:] = float("nan"), float("inf")
    parts = library().ar_expert_parts_workspace
    assert parts(rows, E, N, K, 0) == 0 and parts(rows, E, N, K, 1) == 0
    y = experts.expert_product(x, w, off, dtype=torch.float32)
    want, S = product64(x, w, off)
    assert_sum(y, want, S, K)
    before = normal((E, N, K), 4, torch.float32)
    dw = before.clone()
    experts.expert_gradients(dy, x, w, off, dw=dw, accumulate=True, need_dx=False)
    want, S = weight_gradient64(dy, x, off, E)
    assert_sum(dw, want + before.double(), S + 2 * before.double().abs(), max(counts))
    for e, n in enumerate(counts):
        assert n or torch.equal(dw[e], before[e])
