"""GradClipper against a plain 64-bit form: tensor counts, odd sizes, alignments,
types, special values, streams, graphs.

Tolerances: a thread adds at most a few thousand squares into each of four fp32
accumulators (random rounding: under 2e-6 relative), the rest is added in trees
and in fp64, and the root halves it; so the norm is within 2e-6 and the clipped
values within that plus 2^-23 (fp32) or one rounding, 2^-9 (bf16)."""
import math

import pytest
import torch

from allreduce_reduction_emulated_gb300.clipping import GradClipper

pytestmark = pytest.mark.gpu
NORM_TOL = 2e-6


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def check(grads, max_norm, out=None):
    want = norm64(grads)
    coef = min(1.0, max_norm / (want + 1e-6))
    before = [g.clone() for g in grads]
    c = GradClipper(grads, out=out)
    n0, n1 = c.norm(), c.clip(max_norm)
    assert torch.equal(n0, n1)
    assert abs(float(n1) - want) <= NORM_TOL * want
    for i, (g, b) in enumerate(zip(out if out is not None else grads, before)):
        tol = NORM_TOL * 2 + (2.0 ** -23 if g.dtype == torch.float32 else 2.0 ** -8)
        off = (g.double() - b.double() * coef).abs()
        assert bool((off <= tol * b.double().abs() * coef + 1e-40).all()), i
        if coef == 1.0:
            assert torch.equal(g, b)
    if out is not None:
        assert all(torch.equal(g, b) for g, b in zip(grads, before))


def make(dev, sizes, dtypes, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return [torch.randn(n, device=dev, generator=g).mul_(0.01).to(d) for n, d in zip(sizes, dtypes)]


BOTH = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", BOTH, ids=["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 1000, 8191, 8192, 8193, 16383, 16384, 16385, 100_003, 5_000_001])
def test_one_tensor(dev, n, dtype):
    for max_norm in (1e-3, 1e9):
        check(make(dev, [n], [dtype], n), max_norm)
        grads = make(dev, [n], [dtype], n)
        check(grads, max_norm, [torch.full_like(g, 7.0) for g in grads])


@pytest.mark.parametrize("count", [2, 63, 64, 65, 300, 999, 1000, 1001, 2300])
def test_many_tensors(dev, count):
    """Past the table of one launch; mixed types; empty tensors among them."""
    sizes = [(i * i * 37) % 5000 if i % 11 else 0 for i in range(count)]
    sizes[-1] = 20_001
    dtypes = [BOTH[i % 3 == 0] for i in range(count)]
    check(make(dev, sizes, dtypes, count), 0.25)
    grads = make(dev, sizes, dtypes, count)
    check(grads, 0.25, [torch.zeros_like(g) for g in grads])


@pytest.mark.parametrize("dtype", BOTH, ids=["f32", "bf16"])
@pytest.mark.parametrize("shift_out", [0, 1, 3, 8])
def test_views_at_every_alignment(dev, shift_out, dtype):
    """Gradients and outputs are views of flat buffers; nothing around them changes."""
    sizes = [1, 2, 3, 17, 40_001, 5, 16_390, 9]
    gap = 3
    total = sum(sizes) + gap * len(sizes) + 16
    flat = make(dev, [total], [dtype], 1)[0]
    room = torch.full((total + shift_out,), 5.0, dtype=dtype, device=dev)
    grads, outs, at = [], [], 1
    mark = torch.zeros(total + shift_out, dtype=torch.bool, device=dev)
    for n in sizes:
        grads.append(flat[at:at + n])
        outs.append(room[at + shift_out:at + shift_out + n])
        mark[at + shift_out:at + shift_out + n] = True
        at += n + gap
    check(grads, 0.1, outs)
    assert bool((room[~mark] == 5.0).all())
    whole = flat.clone()
    check(grads, 0.1)
    inside = torch.zeros(total, dtype=torch.bool, device=dev)
    at = 1
    for n in sizes:
        inside[at:at + n] = True
        at += n + gap
    assert torch.equal(flat[~inside], whole[~inside])


@pytest.mark.parametrize("dtype", BOTH, ids=["f32", "bf16"])
def test_special_values(dev, dtype):
    def grads():
        return make(dev, [1000, 30_001], [dtype] * 2, 3)

    g = grads()
    g[1][12345] = math.inf
    n = GradClipper(g).clip(1.0)
    assert float(n) == math.inf
    assert bool(torch.isnan(g[1][12345])) and not bool(g[0].any()) and int(torch.isnan(g[1]).sum()) == 1
    g = grads()
    g[0][5] = math.nan
    n = GradClipper(g).clip(1.0)
    assert math.isnan(float(n)) and all(bool(torch.isnan(x).all()) for x in g)
    g = grads()
    n = GradClipper(g).clip(0.0)
    assert float(n) > 0 and not any(bool(x.any()) for x in g)
    g = [torch.zeros(77, dtype=dtype, device=dev)]
    assert float(GradClipper(g).clip(1.0)) == 0.0 and not bool(g[0].any())
    g = [torch.zeros(0, dtype=dtype, device=dev)]
    assert float(GradClipper(g).clip(1.0)) == 0.0 and float(GradClipper(g).norm()) == 0.0
    g = grads()
    keep = [x.clone() for x in g]
    GradClipper(g).clip(math.inf)
    assert all(torch.equal(a, b) for a, b in zip(g, keep))


def test_more_than_2_to_32_elements(dev):
    n = (1 << 32) + 11
    g = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    for i in (0, 1 << 31, (1 << 32) - 1, n - 1):
        g[i] = 3.0
    norm = GradClipper([g]).clip(0.6)
    assert abs(float(norm) - 6.0) <= 6.0 * NORM_TOL
    want = float(torch.tensor(3.0 * 0.6 / (6.0 + 1e-6)).to(torch.bfloat16))
    assert [float(g[i]) for i in (0, 1 << 31, (1 << 32) - 1, n - 1)] == [want] * 4
    assert int(torch.count_nonzero(g)) == 4


def test_streams_repeats_and_graphs(dev):
    src = make(dev, [70_001, 3, 900], BOTH + [torch.float32], 5)
    outs = [torch.empty_like(g) for g in src]
    c = GradClipper(src, out=outs)
    n = c.clip(0.5)
    want = [o.clone() for o in outs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for how in ("argument", "handle", "current"):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        if how == "current":
            with torch.cuda.stream(side):
                m = c.clip(0.5)
        else:
            m = c.clip(0.5, stream=side if how == "argument" else side.cuda_stream)
        side.synchronize()
        assert torch.equal(m, n) and all(torch.equal(a, b) for a, b in zip(outs, want))
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            m = c.clip(0.5)
    for g, h in zip(src, make(dev, [70_001, 3, 900], BOTH + [torch.float32], 6)):
        g.copy_(h)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.replay()
    side.synchronize()
    assert abs(float(m) - norm64(src)) <= NORM_TOL * norm64(src)
    got = [o.clone() for o in outs]
    n = c.clip(0.5)
    assert torch.equal(m, n) and all(torch.equal(a, b) for a, b in zip(outs, got))


def test_every_call_has_its_own_norm(dev):
    """More calls than one block of results: earlier results stay."""
    g = make(dev, [5000], [torch.float32], 4)
    c = GradClipper(g, out=[torch.empty_like(g[0])])
    first = c.norm()
    kept = []
    for k in range(2 * GradClipper.NORMS + 3):
        kept.append(c.norm())
        g[0].mul_(1.01)
    want = float(first)
    for k, n in enumerate(kept):
        assert abs(float(n) - want * 1.01 ** k) <= 1e-4 * want * 1.01 ** k


def test_clips_again_what_it_clipped(dev):
    """In place, call after call with no host wait: the norm reaches the bound."""
    g = make(dev, [100_000, 33], BOTH, 2)
    c = GradClipper(g)
    norms = [c.clip(2.0 ** -k) for k in range(6)]
    for k in range(1, 6):
        assert abs(float(norms[k]) - 2.0 ** -(k - 1)) <= 1e-4 * 2.0 ** -(k - 1)
