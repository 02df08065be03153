"""Products of rows sorted by expert, and their gradients, against 64 bits."""
import pytest
import torch

from experts_util import assert_sum, product64, ranges, weight_gradient64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from allreduce_reduction_emulated_gb300 import _build

    _build.build()


def normal(shape, seed, dtype=torch.bfloat16, sigma=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=gen) * sigma).to(dtype)


def weights_of(E, N, K, layout, seed=1):
    if layout == "out_in":
        return normal((E, N, K), seed)
    return normal((E, K, N), seed).transpose(1, 2)


def offsets_of(counts, front=0, dtype=torch.int64):
    off = [front]
    for c in counts:
        off.append(off[-1] + c)
    return torch.tensor(off, dtype=dtype, device="cuda")


CASES = [  # counts of rows, in, out
    ([1], 64, 128),
    ([1], 8, 8),
    ([3, 0, 1, 0, 5], 64, 64),
    ([64, 63, 65, 1], 128, 256),
    ([128, 129, 127], 72, 264),
    ([256, 257, 255, 31], 192, 384),
    ([17], 1, 1),
    ([40, 0, 300], 1001, 143),
    ([1, 2], 7, 9),
    ([513, 700, 300, 64], 1024, 2304),      # pairs of blocks
    ([0, 0], 64, 64),
    ([33] * 40, 64, 200),                   # more than 32 experts
    ([2000, 100], 512, 4104),
]
LAYOUTS = ["out_in", "in_out"]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_product(case, dtype, layout):
    from allreduce_reduction_emulated_gb300 import experts

    counts, K, N = CASES[case]
    E, T = len(counts), sum(counts) + 3
    x, w, off = normal((T, K), 2), weights_of(E, N, K, layout), offsets_of(counts, 1)
    # what lies beside the experts' rows must not matter
    x[0], x[-2:] = float("nan"), float("inf")
    y = experts.expert_product(x, w, off, dtype=dtype)
    want, S = product64(x, w, off)
    assert y.dtype == dtype and bool((y[0] == 0).all()) and bool((y[-2:] == 0).all())
    assert_sum(y, want, S, K)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_gradients(case, dtype, layout):
    from allreduce_reduction_emulated_gb300 import experts

    counts, K, N = CASES[case]
    E, T = len(counts), sum(counts) + 3
    x, dy, w, off = normal((T, K), 2), normal((T, N), 3), weights_of(E, N, K, layout), offsets_of(counts, 1)
    x[0], x[-2:] = float("nan"), float("inf")
    dy[0], dy[-2:] = float("inf"), float("nan")
    dx, dw = experts.expert_gradients(dy, x, w, off, dw_dtype=dtype)
    want, S = product64(dy, w.transpose(1, 2), off)
    assert bool((dx[0] == 0).all()) and bool((dx[-2:] == 0).all())
    assert_sum(dx, want, S, N)
    want, S = weight_gradient64(dy, x, off, E)
    assert dw.shape == w.shape and dw.stride() == w.stride() and dw.dtype == dtype
    assert_sum(dw, want, S, max([1] + counts))


def test_infinite_rows_of_the_next_expert():
    """An expert's last slice of rows reaches into the next expert's: nothing of them may come along."""
    from allreduce_reduction_emulated_gb300 import experts

    counts, K, N = [70, 58, 1, 200], 128, 320
    off = offsets_of(counts)
    x, dy, w = normal((sum(counts), K), 5), normal((sum(counts), N), 6), weights_of(4, N, K, "out_in")
    bad = slice(70, 128)
    x[bad], dy[bad] = float("inf"), float("nan")
    _, dw = experts.expert_gradients(dy, x, w, off, dw_dtype=torch.float32)
    want, S = weight_gradient64(dy, x, off, 4)
    for e in (0, 2, 3):
        assert_sum(dw[e], want[e], S[e], counts[e])
    assert bool(torch.isnan(dw[1]).all())


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64], ids=["i32", "i64"])
@pytest.mark.parametrize("off", [[-5, 10, 4, 30, 999], [0, 0, 0, 0, 0], [40, 40, 40, 40, 40], [50, 60, 70, 80, 90],
                                 [30, 20, 10, 5, 0]])
def test_offsets_of_any_values(off, dtype):
    """Clamped, never falling; no row is read or written twice."""
    from allreduce_reduction_emulated_gb300 import experts

    T, K, N = 40, 64, 96
    x, dy, w = normal((T, K), 7), normal((T, N), 8), weights_of(4, N, K, "out_in")
    off = torch.tensor(off, dtype=dtype, device="cuda")
    y = experts.expert_product(x, w, off, dtype=torch.float32)
    want, S = product64(x, w, off)
    assert_sum(y, want, S, K)
    _, dw = experts.expert_gradients(dy, x, w, off)
    want, S = weight_gradient64(dy, x, off, 4)
    assert_sum(dw, want, S, T)


@pytest.mark.parametrize("shift,pad", [(0, 8), (0, 3), (1, 0), (5, 11)])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_strides_and_alignments(shift, pad, layout):
    from allreduce_reduction_emulated_gb300 import experts

    counts, K, N = [100, 3, 77], 120, 200
    T, E = sum(counts) + 4, 3
    off = offsets_of(counts, 2)

    def placed(rows, cols, seed, dtype=torch.bfloat16, fill=None):
        flat = normal((shift + rows * (cols + pad),), seed, dtype)
        if fill is not None:
            flat.fill_(fill)
        return flat, flat[shift:].as_strided((rows, cols), (cols + pad, 1))

    (_, x), (_, dy) = placed(T, K, 1), placed(T, N, 2)
    a, b = (N, K) if layout == "out_in" else (K, N)
    flat = normal((shift + E * (a * (b + pad) + 24),), 3)
    w = flat[shift:].as_strided((E, a, b), (a * (b + pad) + 24, b + pad, 1))
    w = w if layout == "out_in" else w.transpose(1, 2)
    want, S = product64(x, w, off)
    buffer, y = placed(T, N, 4, fill=7.0)
    assert experts.expert_product(x, w, off, out=y) is y
    inside = torch.zeros_like(y, dtype=torch.bool)
    inside[2:2 + sum(counts)] = True
    assert_sum(y[2:-2], want[2:-2], S[2:-2], K)
    assert bool((y[~inside] == 7.0).all()), "rows of no expert are left as they are"
    y.fill_(7.0)
    assert bool((buffer == 7.0).all()), "nothing beside the rows is written"
    bufx, dx = placed(T, K, 5, fill=3.0)
    bufw = torch.full((flat.numel(),), 5.0, device="cuda")
    dw = bufw[shift:].as_strided((E, a, b), (a * (b + pad) + 24, b + pad, 1))
    dw = dw if layout == "out_in" else dw.transpose(1, 2)
    got = experts.expert_gradients(dy, x, w, off, dx=dx, dw=dw)
    assert got[0] is dx and got[1] is dw
    want, S = product64(dy, w.transpose(1, 2), off)
    assert_sum(dx[2:-2], want[2:-2], S[2:-2], N)
    assert bool((dx[:2] == 3.0).all()) and bool((dx[-2:] == 3.0).all())
    want, S = weight_gradient64(dy, x, off, E)
    assert_sum(dw, want, S, 100)
    dx.fill_(3.0)
    dw.fill_(5.0)
    assert bool((bufx == 3.0).all()) and bool((bufw == 5.0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_accumulate(dtype):
    from allreduce_reduction_emulated_gb300 import experts

    counts, K, N = [90, 0, 130], 96, 160
    off = offsets_of(counts)
    x, dy, w = normal((220, K), 1), normal((220, N), 2), weights_of(3, N, K, "out_in")
    before = normal((3, N, K), 9, dtype)
    dw = before.clone()
    dx, got = experts.expert_gradients(dy, x, w, off, dw=dw, accumulate=True, need_dx=False)
    assert dx is None and got is dw
    want, S = weight_gradient64(dy, x, off, 3)
    assert_sum(dw, want + before.double(), S + 2 * before.double().abs(), 130)
    assert torch.equal(dw[1], before[1]), "an expert without rows keeps its own"


def test_repeats_to_the_bit_and_on_other_streams():
    from allreduce_reduction_emulated_gb300 import experts

    counts = [300, 5, 900, 17]
    off = offsets_of(counts)
    x, dy, w = normal((sum(counts), 520), 1), normal((sum(counts), 776), 2), weights_of(4, 776, 520, "out_in")
    y = experts.expert_product(x, w, off)
    dx, dw = experts.expert_gradients(dy, x, w, off)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams * 2:                       # several calls on their way at once
        y2 = experts.expert_product(x, w, off, stream=s)
        got.append((y2, *experts.expert_gradients(dy, x, w, off, stream=s.cuda_stream)))
    torch.cuda.synchronize()
    for a in got:
        assert all(torch.equal(p, q) for p, q in zip(a, (y, dx, dw)))


def test_captured_and_replayed():
    from allreduce_reduction_emulated_gb300 import experts

    counts = [40, 90, 70]
    off = offsets_of(counts)
    x, dy = normal((200, 100), 1), normal((200, 136), 2)        # x is laid out anew in every replay
    w = weights_of(3, 136, 100, "out_in")
    y = torch.empty(200, 136, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        experts.expert_product(x, w, off, out=y)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            experts.expert_product(x, w, off, out=y)
            dx, dw = experts.expert_gradients(dy, x, w, off)
    for seed, counts in ((5, [40, 90, 70]), (6, [200, 0, 0]), (7, [0, 1, 150])):
        x.copy_(normal(x.shape, seed))
        off.copy_(offsets_of(counts))
        y.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        want, S = product64(x, w, off)
        assert_sum(y, want, S, 100)
        want, S = weight_gradient64(dy, x, off, 3)
        assert_sum(dw, want, S, 200)


def test_nothing_to_do():
    from allreduce_reduction_emulated_gb300 import experts

    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    off0, off3 = offsets_of([]), offsets_of([0, 0, 0])
    assert experts.expert_product(e(0, 64), e(3, 32, 64), off3).shape == (0, 32)
    assert experts.expert_product(e(5, 64), e(3, 0, 64), off3).shape == (5, 0)
    assert bool((experts.expert_product(e(5, 0), e(3, 8, 0), offsets_of([1, 2, 2])) == 0).all())
    assert bool((experts.expert_product(e(5, 64), e(0, 8, 64), off0) == 0).all())
    dx, dw = experts.expert_gradients(e(0, 32), e(0, 64), e(3, 32, 64), off3)
    assert dx.shape == (0, 64) and bool((dw == 0).all())
    dx, dw = experts.expert_gradients(e(4, 32), e(4, 64), e(0, 32, 64), off0)
    assert bool((dx == 0).all()) and dw.shape == (0, 32, 64)


def test_more_rows_than_a_tile_of_one_expert_and_many_experts():
    from allreduce_reduction_emulated_gb300 import experts

    counts = [i % 7 for i in range(1024)]
    off = offsets_of(counts)
    x, w = normal((sum(counts), 64), 1), weights_of(1024, 64, 64, "out_in")
    y = experts.expert_product(x, w, off, dtype=torch.float32)
    want, S = product64(x, w, off)
    assert_sum(y, want, S, 64)
    _, dw = experts.expert_gradients(y.to(torch.bfloat16), x, w, off)
    want, S = weight_gradient64(y.to(torch.bfloat16), x, off, 1024)
    assert_sum(dw, want, S, 16)
    x, w = normal((20000, 256), 3), weights_of(1, 640, 256, "in_out")
    y = experts.expert_product(x, w, offsets_of([20000]))
    want, S = product64(x, w, offsets_of([20000]))
    assert_sum(y, want, S, 256)
    _, dw = experts.expert_gradients(y, x, w, offsets_of([20000]), dw_dtype=torch.float32, need_dx=False)
    want, S = weight_gradient64(y, x, offsets_of([20000]), 1)
    assert_sum(dw, want, S, 20000)
