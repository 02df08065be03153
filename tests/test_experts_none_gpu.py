"""A product without experts through the C entry, with more workspace than it needs: rows of no expert only."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from allreduce_reduction_emulated_gb300 import _build, library

    _build.build()
    return library()


@pytest.mark.parametrize("zero_rest", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("out", [64, 130])
def test_no_experts_and_a_large_workspace(lib, dtype, zero_rest, out):
    from allreduce_reduction_emulated_gb300 import AR_BFLOAT16, AR_FLOAT32, AR_SUCCESS

    rows, features = 9, 8192                                     # a sum long enough to be split into parts
    x = torch.ones(rows, features, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0], device="cuda")
    need = lib.ar_expert_parts_workspace(rows, 1, out, features, 0)
    assert need > 0
    space = torch.full((need + 256,), 1.5, dtype=torch.float32, device="cuda")   # what another call may have left
    y = torch.full((rows, out), 3.0, dtype=dtype, device="cuda")
    st = lib.ar_expert_product(x.data_ptr(), rows, features, None, 0, out, features, 0, 0, 0, off.data_ptr(), 8,
                               y.data_ptr(), out, AR_FLOAT32 if dtype == torch.float32 else AR_BFLOAT16, zero_rest,
                               space.data_ptr(), space.numel() * 4, torch.cuda.current_stream().cuda_stream)
    assert st == AR_SUCCESS
    assert bool((y == (0.0 if zero_rest else 3.0)).all())
    assert bool((space == 1.5).all())
