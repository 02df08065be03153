"""Orthogonalised updates where single elements, single directions or sizes matter, against 64 bits."""
import pytest
import torch

from orthogonal_util import assert_update, update64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from allreduce_reduction_emulated_gb300 import _build

    _build.build()


@pytest.mark.parametrize("tall", [False, True], ids=["wide", "tall"])
@pytest.mark.parametrize("shape", [(2, 21), (100, 128), (130, 600)], ids=str)   # whole in a block twice, in tiles
def test_an_element_of_b_next_to_zero(shape, tall):
    """B = a I - A with B_11 of 3 * 2^-25 as it is held, between two values of fp16, beside B_10 of -16.

    The rows' squares add up to 1 exactly (21 columns of 2^-k, three of each, and 2^-7), so that X is exact in fp16:
    A_00 = 1 - 4^-7, A_10 = 2^-8, A_11 = 4^-7, and with a = 4^-7 (1 + 3 * 2^-23), held times 2^12, row 1 of the result is
    -2^-8 of row 0 but for 2^-30 of row 1.  Its powers of two are exact in bf16, too; rounding B_10 costs at most 2^-11 and
    A_00 2^-14.  So row 1 is within 2^-10 of itself, whatever becomes of B_11."""
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    g = torch.zeros(shape, device="cuda")
    g[0, :21] = torch.tensor([2.0 ** -k for k in range(1, 8) for _ in range(3)])
    g[1, 0] = 2.0 ** -7
    assert float(g.double().square().sum()) == 1.0
    kw = dict(steps=1, coefficients=(4.0 ** -7 * (1 + 3 * 2.0 ** -23), -1.0, 0.0), eps=0.0)
    want = update64(g, **kw)[0]
    (u,) = Orthogonalizer([g.t().contiguous() if tall else g], **kw).update()
    u = u.t() if tall else u
    for row in range(2):
        off = (u[row].double() - want[row]).norm() / want[row].norm()
        assert float(off) <= 2.0 ** -10 + (2.0 ** -8 if row == 0 else 0.0), (row, float(off))
    assert bool((u[2:] == 0).all())
