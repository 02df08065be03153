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


# ------------------------------------------------------------------ a tolerance from each matrix' own singular values

def poly(t, coefficients, times):
    a, b, c = coefficients
    for _ in range(times):
        t = t * (a + b * t ** 2 + c * t ** 4)
    return t


def growth(s, reach, length, coefficients, times):
    """How far `times` steps carry an error of matrices with singular values s (stack, n), long side `length`: the error of
    the result over that of the matrix (2-norms, Frobenius), if it lies evenly in all directions.  In the singular vectors'
    basis an error's element (i, j) goes on times (p_i - p_j) / (s_i - s_j) as far as it is symmetric, (p_i + p_j) /
    (s_i + s_j) as far as it is not, times p' on the diagonal and times p_i / s_i outside the square.  The singular
    values themselves may be off by `reach` (stack): the largest in that range counts."""
    n = s.shape[1]
    at = torch.linspace(-1, 1, 7, dtype=s.dtype)
    t = (s[:, :, None] + reach[:, None, None] * at).clamp_min(1e-12)         # (stack, n, 7)
    p = poly(t, coefficients, times)
    x, y, px, py = t[:, :, None, :, None], t[:, None, :, None, :], p[:, :, None, :, None], p[:, None, :, None, :]
    apart = (x - y).abs()
    chord = torch.where(apart > 1e-5 * (x + y), (px - py).abs() / apart.clamp_min(1e-30), torch.zeros(()).double())
    d = torch.maximum(chord, (px + py).abs() / (x + y)).flatten(3).amax(3)    # (stack, n, n)
    step = t * 1e-6
    slope = ((poly(t + step, coefficients, times) - p) / step).abs().amax(2)
    d = torch.maximum(d, torch.diag_embed(slope))
    outside = (length - n) * (p / t).abs().amax(2).square().sum(1)
    return ((d.square().sum((1, 2)) + outside) / (n * length)).sqrt()


def tolerance(g, coefficients=(3.4445, -4.7750, 2.0315), steps=5):
    """What the result may be off by (2-norm, Frobenius; one per matrix of the stack).

    X, A = X X^T and B = a I + b A + c A^2 are held in fp16, each element off by half a step, 2^-11 of its value, at most
    and 2^-11 / sqrt(3) in the mean square.  X's error goes on by `growth` of the steps left; element (i, j)
    of A's, in the singular vectors' basis, comes into B times b + c (s_i^2 + s_j^2), B's own beside it, and both times s_j into
    the next X.  The roundings are independent, so their squares add up.  Six times that: an error can lie in one direction only, which for 2 x 2 makes it sqrt(4) larger, and be at
    its most, sqrt(3); six standard deviations where there are many.  fp32 sums and the norm, some 2^-20, are within
    the factor 1.02.  The result is rounded to bf16 once: 2^-8 of each element."""
    a, b, c = coefficients
    unit = 2.0 ** -11 / 3 ** 0.5
    x = g.double().cpu()
    x = x if x.shape[-2] <= x.shape[-1] else x.transpose(-1, -2)
    length = x.shape[-1]
    size = lambda m: m.flatten(1).norm(dim=1)  # noqa: E731
    x = x / size(x)[:, None, None]
    total, carried = torch.zeros(len(x)).double(), torch.zeros(len(x)).double()   # squares
    for k in range(steps):
        s = torch.linalg.svdvals(x)
        A = x @ x.transpose(-1, -2)
        B = b * A + c * A @ A + a * torch.eye(A.shape[-1], dtype=x.dtype)
        now = (unit * size(x)) ** 2
        carried = carried + now
        total = total + now * growth(s, 6 * carried.sqrt(), length, coefficients, steps - k) ** 2
        pair = b + c * (s[:, :, None] ** 2 + s[:, None, :] ** 2)
        into = (unit * size(A)) ** 2 * (pair * s[:, None, :]).square().mean((1, 2)) + (unit * size(B)) ** 2 * s.square().mean(1)
        carried = carried * growth(s, 6 * carried.sqrt(), length, coefficients, 1) ** 2 + into
        x = B @ x
        total = total + into * growth(torch.linalg.svdvals(x), 6 * carried.sqrt(), length, coefficients, steps - 1 - k) ** 2
    total = 6 * 1.02 * total.sqrt()
    return total + 2.0 ** -8 * (size(x) + total)


@pytest.mark.parametrize("shape", [(2, 2), (2, 3), (3, 2), (3, 3), (4, 4), (13, 2), (2, 27), (5, 4), (8, 8), (3, 300),
                                   (2, 700), (700, 4)], ids=str)
def test_short_sides(shape):
    """Two or three directions: a weak one has few others to share the roundings with."""
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    g = torch.randn(256, *shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(sum(shape)))
    (u,) = Orthogonalizer([g]).update()
    off = (u.double() - update64(g)[0]).flatten(1).norm(dim=1).cpu()
    most = tolerance(g)
    assert bool((off <= most).all()), float((off / most).max())


def test_large_and_of_several_shapes():
    """Tiles of 256 columns by pairs of blocks, tall matrices beside wide ones, with momentum."""
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    shapes = [(1300, 2700), (2600, 1100), (2, 1536, 1536), (1281, 4100), (2049, 1025), (40, 70), (1100, 1030)]
    gen = torch.Generator(device="cuda").manual_seed(3)
    grads = [torch.randn(s, device="cuda", generator=gen) * 1e-3 for s in shapes]
    momentum = [torch.randn(s, device="cuda", generator=gen) * 1e-3 for s in shapes]
    want = [update64(g, m) for g, m in zip(grads, momentum)]
    got = Orthogonalizer(grads, momentum=momentum).update()
    for u, m, (w, m64), g in zip(got, momentum, want, grads):
        # beta, beta m and the sum: 3 roundings of 2^-24 of at most |m| + |g|
        assert bool(((m - m64).abs() <= 3 * 2.0 ** -24 * (m64.abs() + 2 * g.abs())).all())
        assert_update(u, w)


def test_the_same_bits_alone_and_among_others():
    """What else is on the list changes how tiles are cut; which products a sum adds up, and in which order, stays."""
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    gen = torch.Generator(device="cuda").manual_seed(4)
    for shape in ((384, 512), (500, 260), (3, 200, 777)):
        g = torch.randn(shape, device="cuda", generator=gen)
        alone = Orthogonalizer([g]).update()[0]
        for others in ((1, 512, 512), (10, 512, 512), (2, 300, 1200)):
            o = torch.randn(others, device="cuda", generator=gen)
            assert torch.equal(alone, Orthogonalizer([g, o]).update()[0])
            assert torch.equal(alone, Orthogonalizer([o, g]).update()[1])
