"""Handles made on one stream and first used on another: their own memory may have belonged to tensors that
kernels on their way still use."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BUSY = 400_000_000   # cycles: a fifth of a second


@pytest.fixture(scope="module", autouse=True)
def built():
    from allreduce_reduction_emulated_gb300 import _build

    _build.build()


def freed_while_used(bytes_):
    """Copies, at the end of a queue, of tensors of so many bytes that are freed by now: what is allocated next is theirs."""
    old = [torch.full((bytes_,), 5, dtype=torch.uint8, device="cuda") for _ in range(32)]
    copies = [torch.empty_like(t) for t in old]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for c, t in zip(copies, old):
        c.copy_(t)
    return copies


def first_used_elsewhere(make, use, bytes_):
    s = torch.cuda.Stream()
    copies = freed_while_used(bytes_)
    got = use(make(), s)
    torch.cuda.synchronize()
    assert all(bool((c == 5).all()) for c in copies), "the memory is another tensor's until its kernels are done"
    return got


def test_orthogonalizer():
    from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer

    gen = torch.Generator(device="cuda").manual_seed(1)
    g = torch.randn(1024, 2048, device="cuda", generator=gen)
    out = [torch.empty(g.shape, dtype=torch.bfloat16, device="cuda")]
    probe = Orthogonalizer([g], out=out)
    want = probe.update()[0].clone()
    bytes_ = probe._workspace.numel()
    del probe
    got = first_used_elsewhere(lambda: Orthogonalizer([g], out=out), lambda o, s: o.update(stream=s)[0], bytes_)
    assert torch.equal(got, want)


def test_clipper():
    from allreduce_reduction_emulated_gb300.clipping import GradClipper

    g = [torch.ones(1 << 22, device="cuda")]
    probe = GradClipper(g)
    bytes_ = probe._workspace.numel()
    probe.norm()                        # (a kernel's first launch may wait for the GPU)
    del probe
    assert float(first_used_elsewhere(lambda: GradClipper(g), lambda c, s: c.norm(stream=s), bytes_)) == 2048.0
    got = first_used_elsewhere(lambda: GradClipper(g), lambda c, s: c.clip(1.0, stream=s), bytes_)
    assert float(got) == 2048.0 and float(g[0][0]) == 1 / 2048
