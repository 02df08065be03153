"""Whose memory the norms of GradClipper are: the pool of the call's stream, one
norm for one call, for as long as anything may write it."""
import sys
import threading

import pytest
import torch

from allreduce_reduction_emulated_gb300.clipping import GradClipper

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def pool_of(t):
    """The stream whose memory pool a tensor's memory is from."""
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


@pytest.mark.parametrize("given", [None, "object", "handle"])
@pytest.mark.parametrize("call", ["home", "other"])
@pytest.mark.parametrize("current", ["home", "other"])
def test_norms_are_from_the_pool_of_the_calls_stream(dev, current, call, given):
    home, other = torch.cuda.Stream(), torch.cuda.Stream()
    on = {"home": home, "other": other}
    grads = [torch.full((1000,), 2.0, device=dev)]
    torch.cuda.synchronize()
    with torch.cuda.stream(home):
        clipper = GradClipper(grads)
    stream = {None: None, "object": on[call], "handle": on[call].cuda_stream}[given]
    want = on[current if given is None else call]
    with torch.cuda.stream(on[current]):
        norms = [clipper.norm(stream=stream), clipper.clip(1e9, stream=stream)]
    torch.cuda.synchronize()
    for n in norms:
        assert abs(float(n) - 4000 ** 0.5) < 1e-4
        assert pool_of(n) == want.cuda_stream


@pytest.mark.parametrize("how", ["current", "object", "handle"])
def test_a_captured_call_keeps_its_norm(dev, how):
    """A graph captured on the clipper's own stream writes its norm in every replay: no
    other tensor may ever get that memory while the clipper is there."""
    home = torch.cuda.Stream()
    g = torch.full((1000,), 2.0, device=dev)
    torch.cuda.synchronize()
    with torch.cuda.stream(home):
        clipper = GradClipper([g])
        clipper.norm()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=home):
            norm = clipper.norm(stream={"current": None, "object": home, "handle": home.cuda_stream}[how])
        graph.replay()
        home.synchronize()
        assert abs(float(norm) - 4000 ** 0.5) < 1e-4
        at = norm.data_ptr()
        del norm
        for _ in range(GradClipper.NORMS + 2):        # a new block: the one before is given back
            clipper.norm()
        home.synchronize()
        others = [torch.full((n,), -7.0, device=dev) for n in (128, 256, 1024) for _ in range(256)]
        assert not [t for t in others if t.data_ptr() <= at < t.data_ptr() + 4 * t.numel()]
        graph.replay()
        home.synchronize()
        assert all(bool((t == -7.0).all()) for t in others)


def test_threads_get_norms_of_their_own(dev):
    """Calls from several threads on one stream, which runs them one after the other."""
    clipper = GradClipper([torch.full((1000,), 2.0, device=dev)])
    calls, threads = 5 * GradClipper.NORMS, 4
    got = [[] for _ in range(threads)]
    start = threading.Barrier(threads)

    def work(mine):
        start.wait()
        for _ in range(calls):
            mine.append(clipper.norm())

    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        each = [threading.Thread(target=work, args=(mine,)) for mine in got]
        for t in each:
            t.start()
        for t in each:
            t.join()
    finally:
        sys.setswitchinterval(before)
    torch.cuda.synchronize()
    norms = [n for mine in got for n in mine]
    assert len(norms) == calls * threads
    assert len({n.data_ptr() for n in norms}) == len(norms)
    assert all(abs(float(n) - 4000 ** 0.5) < 1e-4 for n in norms)


def test_calls_from_threads_do_not_mix(dev):
    """Clipping in place from several threads on one stream: each call takes the norm that the call
    before it on the stream has left.  With bound and eps 1e4 a call makes n to n / (1 + n / 1e4), so
    the reciprocals of the norms grow by 1e-4 from call to call.  The GPU is behind, so that launches wait."""
    g = torch.full((8_000_000,), 8e6 ** -0.5, device=dev)
    clipper = GradClipper([g])
    calls, threads = 3000, 4
    got = [[] for _ in range(threads)]
    start = threading.Barrier(threads)

    def work(mine):
        start.wait()
        for _ in range(calls):
            mine.append(clipper.clip(1e4, eps=1e4))

    each = [threading.Thread(target=work, args=(mine,)) for mine in got]
    for t in each:
        t.start()
    for t in each:
        t.join()
    torch.cuda.synchronize()
    inverse = sorted(1.0 / float(n) for mine in got for n in mine)
    assert abs(inverse[0] - 1.0) < 1e-5
    # a call's norm and coefficient each round a few times: 2e-6 of an inverse of at most 2.2
    assert all(abs(b - a - 1e-4) < 1e-5 for a, b in zip(inverse, inverse[1:]))


@pytest.mark.parametrize("which", ["grads", "out"])
def test_memory_of_replaced_tensors_stays_the_clippers(dev, which):
    """A tensor whose storage is replaced (t.data = ...): the clipper goes on with the memory that it was
    given, which nothing else may get meanwhile."""
    n = 1 << 20
    g, o = torch.full((n,), 2.0, device=dev), torch.zeros(n, device=dev)
    clipper = GradClipper([g], out=[o] if which == "out" else None)
    t = o if which == "out" else g
    at = t.data_ptr()
    t.data = torch.zeros(8, device=dev)
    others = [torch.full((n,), -7.0, device=dev) for _ in range(8)]
    assert at not in [x.data_ptr() for x in others]
    assert abs(float(clipper.clip(1.0)) - 2.0 * n ** 0.5) < 1e-2
    assert all(bool((x == -7.0).all()) for x in others)
