"""Orthogonalised updates against 64 bits."""
import pytest
import torch

from orthogonal_util import assert_update, update64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from allreduce_reduction_emulated_gb300 import _build

    _build.build()


def gradient(shape, seed, dtype=torch.float32, sigma=1e-3):
    """Noise and a few strong directions."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    *lead, m, n = shape
    g = torch.randn(shape, device="cuda", generator=gen)
    g += 0.2 * torch.randn(*lead, m, 4, device="cuda", generator=gen) @ torch.randn(*lead, 4, n, device="cuda", generator=gen)
    return (g * sigma).to(dtype)


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 2), (16, 16), (8, 64), (64, 8), (33, 65), (65, 33), (128, 128), (96, 1000),
          (1000, 96), (127, 129), (256, 256), (300, 200), (200, 300), (257, 600), (513, 512), (3, 128, 256), (4, 260, 130),
          (2, 2, 40, 72), (640, 1920), (1920, 640)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_update(shape, dtype):
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    g = gradient(shape, 1, dtype)
    kept = g.clone()
    (u,) = Orthogonalizer([g]).update()
    assert u.dtype == torch.bfloat16 and u.shape == g.shape and torch.equal(g, kept)
    assert_update(u, update64(g)[0])


@pytest.mark.parametrize("nesterov", [True, False])
def test_momentum_over_three_steps(nesterov):
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    shapes = [(64, 200), (3, 130, 70), (65, 33)]
    grads = [gradient(s, i, torch.bfloat16) for i, s in enumerate(shapes)]
    momentum = [torch.zeros(s, device="cuda") for s in shapes]
    ortho = Orthogonalizer(grads, momentum=momentum, beta=0.9, nesterov=nesterov)
    want = [torch.zeros(s, dtype=torch.float64, device="cuda") for s in shapes]
    size = [torch.zeros(s, dtype=torch.float64, device="cuda") for s in shapes]
    for step in range(3):
        for i, g in enumerate(grads):
            g.copy_(gradient(g.shape, 10 * step + i, torch.bfloat16))
        updates = ortho.update()
        assert updates is ortho.out
        for g, u, m, k in zip(grads, updates, momentum, range(3)):
            w, want[k] = update64(g, want[k], 0.9, nesterov)
            # Every step rounds beta, beta m and the sum: 2^-24 each of at most size = 0.9 size + |g|, which terms that
            # cancel leave above |m|; what the steps before were off by falls by beta.  Three steps: 9 times 2^-24.
            size[k] = 0.9 * size[k] + g.double().abs()
            assert bool(((m - want[k]).abs() <= 9 * 2.0 ** -24 * size[k]).all())
            assert_update(u, w)


@pytest.mark.parametrize("kw", [dict(steps=1), dict(steps=2), dict(steps=9), dict(coefficients=(1.5, -0.5, 0.0)),
                                dict(coefficients=(2.0, -1.5, 0.5), steps=12), dict(scale=0.2), dict(eps=1e-3)], ids=str)
def test_parameters(kw):
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    g = [gradient((100, 250), 1), gradient((250, 100), 2)]
    for got, x in zip(Orthogonalizer(g, **kw).update(), g):
        # few steps leave small singular values small: eps and the fp16 of the first X are all that counts
        assert_update(got, update64(x, **kw)[0])


def test_scale_by_shape_and_list():
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    g = [gradient((300, 75), 1), gradient((75, 300), 2)]
    a, b = Orthogonalizer(g, scale="shape").update()
    assert_update(a, update64(g[0], scale=2.0)[0])
    assert_update(b, update64(g[1])[0])
    a, b = Orthogonalizer(g, scale=[-1.0, 0.5]).update()
    assert_update(a, update64(g[0], scale=-1.0)[0])
    assert_update(b, update64(g[1], scale=0.5)[0])


@pytest.mark.parametrize("sigma", [1e-18, 1e-9, 1.0, 1e5, 1e12])
def test_sizes_of_values(sigma):
    """Only beside eps does the size of the gradient matter."""
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    g = gradient((90, 160), 3, sigma=sigma)
    for eps in (1e-7, 0.0):
        assert_update(Orthogonalizer([g], eps=eps).update()[0], update64(g, eps=eps)[0])


def test_strong_directions():
    """Singular values over a range of 300, one matrix of rank one, one of a single element."""
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    q, _ = torch.linalg.qr(torch.randn(200, 200, device="cuda", dtype=torch.float64))
    r, _ = torch.linalg.qr(torch.randn(320, 200, device="cuda", dtype=torch.float64))
    s = torch.logspace(0, -2.5, 200, device="cuda", dtype=torch.float64)
    full = ((q * s) @ r.t()).float()
    one = (q[:, :1] @ r[:, :1].t()).float()
    spike = torch.zeros(200, 320, device="cuda")
    spike[17, 130] = -3.0
    got = Orthogonalizer([full, one, spike]).update()
    # Rounding the first X to fp16 puts 2.8e-4 of its 2-norm, 4.17, into 200 directions: 8.3e-5 to each, which is relative
    # to the direction's singular value s from then on.  Over s from 1 to 10^-2.5, equally far apart in their
    # logarithm, the mean of 1 / s^2 is (10^5 - 1) / (5 ln 10) = 8686: 93 * 8.3e-5 = 7.7e-3.  In the next step s has
    # grown at least as much as the 2-norm, so its rounding adds at most as much, and later ones, as the
    # range closes, less and less: 7.7e-3 sqrt(2), and bf16's 2.3e-3.
    assert_update(got[0], update64(full)[0], 7.7e-3 * 2 ** 0.5 + 2.3e-3)
    assert_update(got[2], update64(spike)[0])
    # Of a matrix of rank one the other directions hold what rounding puts there.  They grow by 3.4445 a step: fp16 adds
    # 2.8e-4 of the 2-norm, 1 of the first X and at most 1.2 of the later ones, to X and to its increment.
    w, grown = update64(one)[0], 3.4445 ** torch.arange(6).double()
    assert float((got[1].double() - w).norm()) <= 2.8e-4 * float(grown[5] + 1.2 * grown[:5].sum()) + 5e-3


def test_zeros_and_what_is_not_finite():
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    g = gradient((4, 70, 90), 1)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    g[3, 69, 89] = float("inf")
    for eps in (1e-7, 0.0):
        (u,) = Orthogonalizer([g], eps=eps).update()
        assert_update(u[0], update64(g[0])[0])
        assert bool((u[1] == 0).all()) and bool(torch.isnan(u[2:]).all())


def test_many_shapes_and_tensors():
    """More shapes than one group of launches takes, more tensors than that too, empty ones between."""
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    shapes = [(8 + i % 40, 200 - 3 * (i % 40)) for i in range(300)] + [(0, 5), (0, 3, 4), (5, 0)]
    g = [gradient(s, i) for i, s in enumerate(shapes)]
    m = [torch.zeros_like(x) for x in g]
    for u, x in zip(Orthogonalizer(g, momentum=m).update(), g):
        if x.numel():
            assert_update(u, update64(x)[0])


def test_alignments_and_in_place():
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    m, n = 72, 104
    flat = torch.zeros(3 * m * n + 40, device="cuda")
    g = [flat[1 + i * (m * n + 3):][:m * n].view(m, n) for i in range(3)]
    for i, x in enumerate(g):
        x.copy_(gradient((m, n), i))
    outs = torch.full((3 * m * n + 40,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = [outs[5 + i * (m * n + 7):][:m * n].view(m, n) for i in range(3)]
    Orthogonalizer(g, out=out).update()
    for x, u in zip(g, out):
        assert_update(u, update64(x)[0])
        u.fill_(9.0)
    assert bool((outs == 9.0).all())
    x = gradient((m, n), 7, torch.bfloat16)
    want = update64(x)[0]
    assert Orthogonalizer([x], out=[x]).update()[0] is x
    assert_update(x, want)


def test_repeats_to_the_bit_on_streams_and_replayed():
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    g = [gradient((6, 200, 330), 1), gradient((700, 260), 2)]
    ortho = Orthogonalizer(g)
    want = [u.clone() for u in ortho.update()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ortho.update(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, ortho.out))
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            ortho.update()
    g2 = [gradient((6, 200, 330), 5), gradient((700, 260), 6)]
    for a, b in zip(g, g2):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    got = [u.clone() for u in ortho.out]
    assert not torch.equal(got[0], want[0])
    assert all(torch.equal(a, b) for a, b in zip(got, Orthogonalizer(g2).update()))


def test_alone_and_among_others_alike():
    """What else is on the list changes the tiles' sizes, not the values they are rounded from."""
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    g = gradient((384, 512), 1)
    others = [gradient((40, 512, 512), 2)]
    a = Orthogonalizer([g]).update()[0]
    b = Orthogonalizer([g] + others).update()[0]
    assert_update(a, update64(g)[0])
    assert_update(b, update64(g)[0])
