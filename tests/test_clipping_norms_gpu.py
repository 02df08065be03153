"""Whose memory the norms of GradClipper are: the pool of the call's stream, one
norm for one call, for as long as anything may write it."""
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
