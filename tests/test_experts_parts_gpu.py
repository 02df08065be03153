"""Long sums of few tiles, which are split into parts, and operands at odd strides with experts without rows."""
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


def weights_of(E, N, K, layout):
    return normal((E, N, K), 1) if layout == "out_in" else normal((E, K, N), 1).transpose(1, 2)


def k_of(k):
    """assert_sum counts an addition for every 16; the 16 parts at most are as many more."""
    return k + 16 * 16


def parts(rows, E, N, K, of_weights):
    from allreduce_reduction_emulated_gb300 import library

    return library().ar_expert_parts_workspace(rows, E, N, K, of_weights)


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("off,rows,N,K", [
    ([0, 2, 2, 3, 5], 5, 200, 8200),
    ([4, 4, 9], 30, 72, 4097),
    ([0, 130], 131, 129, 65536 + 40),
    ([1, 17, 90], 93, 640, 5120),
    ([7, 7], 7, 64, 16384),          # rows of no expert alone
])
def test_products_in_parts(off, rows, N, K, dtype, layout):
    from allreduce_reduction_emulated_gb300 import experts

    E = len(off) - 1
    x, w, off = normal((rows, K), 2), weights_of(E, N, K, layout), torch.tensor(off, device="cuda")
    assert parts(rows, E, N, K, 0) > 0
    y = experts.expert_product(x, w, off, dtype=dtype)
    want, S = product64(x, w, off)
    assert_sum(y, want, S, k_of(K))
    wide = torch.full((rows + 2, N + 9), 3.0, device="cuda", dtype=dtype)
    out = wide[1:-1, 5:5 + N]
    experts.expert_product(x, w, off, out=out)
    a, b = int(off[0]), int(off[-1])
    assert torch.equal(out[a:b], y[a:b])
    out[a:b] = 3.0
    assert bool((wide == 3.0).all()), "rows of no expert and what lies around are left as they are"
    # the same function from the other side: dx
    dx, _ = experts.expert_gradients(x, y.bfloat16(), w.transpose(1, 2), off, need_dw=False)
    want, S = product64(x, w, off)
    assert_sum(dx, want, S, k_of(K))


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts,N,K", [
    ([8000, 8000], 264, 163),
    ([9000], 64, 128),
    ([1, 9999, 0, 63], 130, 72),     # parts of a slice, of none
    ([20011], 1, 7),
])
def test_weight_gradients_in_parts(counts, N, K, dtype, layout):
    from allreduce_reduction_emulated_gb300 import experts

    E, rows = len(counts), sum(counts) + 9
    ends = torch.tensor([0] + counts).cumsum(0) + 4
    off = ends.int().cuda()
    x, dy, w = normal((rows, K), 3), normal((rows, N), 4), weights_of(E, N, K, layout)
    x[:4] = float("inf")             # of no expert
    dy[-5:] = float("nan")
    assert parts(rows, E, N, K, 1) > 0
    _, dw = experts.expert_gradients(dy, x, w, off, dw_dtype=dtype, need_dx=False)
    want, S = weight_gradient64(dy, x, off, E)
    assert_sum(dw, want, S, k_of(rows))
    before = normal((E, N, K), 5, dtype)
    more = before.clone()
    if layout == "in_out":
        more = before.transpose(1, 2).clone(memory_format=torch.contiguous_format).transpose(1, 2)
    experts.expert_gradients(dy, x, w, off, dw=more, accumulate=True, need_dx=False)
    assert_sum(more, want + before.double(), S + 2 * before.double().abs(), k_of(rows))
    for e, n in enumerate(counts):
        assert n or torch.equal(more[e], before[e])


def test_parts_repeat_to_the_bit_and_replay():
    from allreduce_reduction_emulated_gb300 import experts

    x, dy, w = normal((6000, 104), 1), normal((6000, 200), 2), weights_of(2, 200, 104, "out_in")
    long, heavy = normal((9, 8192), 3), weights_of(2, 64, 8192, "in_out")
    off, few = torch.tensor([0, 2500, 6000], device="cuda"), torch.tensor([0, 3, 9], device="cuda")

    def run():
        return experts.expert_product(long, heavy, few), *experts.expert_gradients(dy, x, w, off)

    first = run()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for s in streams * 3:
        with torch.cuda.stream(s):
            got.append(run())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    long.mul_(2)
    dy.mul_(2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b * 2) for a, b in zip(held, first))


def test_without_the_workspace_for_parts():
    """The C entry with the operands' workspace alone: whole sums."""
    from allreduce_reduction_emulated_gb300 import AR_FLOAT32, AR_SUCCESS, library

    x, w, off = normal((9, 8192), 3), normal((2, 64, 8192), 4), torch.tensor([0, 3, 9], device="cuda")
    want, S = product64(x, w, off)
    n = parts(9, 2, 64, 8192, 0)
    for bytes_ in (0, n - 4, n, n + 16):
        space = torch.full((bytes_ + 64,), 77, dtype=torch.uint8, device="cuda")
        y = torch.empty(9, 64, device="cuda")
        assert library().ar_expert_product(x.data_ptr(), 9, 8192, w.data_ptr(), 2, 64, 8192, 64 * 8192, 8192, 1,
                                           off.data_ptr(), 8, y.data_ptr(), 64, AR_FLOAT32, 0, space.data_ptr(), bytes_,
                                           torch.cuda.current_stream().cuda_stream) == AR_SUCCESS
        assert_sum(y, want, S, k_of(8192))
        assert bool((space[bytes_:] == 77).all())


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("shift", [0, 1, 3, 6])
def test_packed_weights_of_experts_without_rows(layout, shift):
    """Odd strides: what has no rows is not laid out, and may hold anything."""
    from allreduce_reduction_emulated_gb300 import experts

    E, N, K = 9, 77, 131
    flat = torch.full((E * (N * K + 5) + shift,), float("nan"), device="cuda", dtype=torch.bfloat16)
    w = flat[shift:].as_strided((E, N, K), (N * K + 5, K, 1) if layout == "out_in" else (N * K + 5, 1, N), shift)
    full = torch.tensor([0, 0, 7, 7, 5, 9, 9, 30, 30, 41], device="cuda")   # (5: as 7)
    has = [1, 4, 6, 8]
    w[has] = normal((4, N, K), 1)
    x = normal((44, K + 3), 2)[:, shift % 3:shift % 3 + K]
    y = experts.expert_product(x, w, full, dtype=torch.float32)
    clean = torch.where(torch.isnan(w), torch.zeros_like(w), w)
    want, S = product64(x, clean, full)
    assert_sum(y, want, S, K)
