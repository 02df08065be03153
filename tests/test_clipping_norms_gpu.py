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
