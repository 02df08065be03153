"""Refusals of the training operators' binding that need no GPU."""
import pytest
import torch

import allreduce_reduction_emulated_gb300 as ar
from allreduce_reduction_emulated_gb300 import clipping
from test_train_abi import CudaLike, refused


@pytest.mark.parametrize("what", [None, 1.0, [0.0], "g"], ids=["None", "number", "list", "text"])
def test_clipper_refuses_what_is_not_a_tensor(what):
    """A parameter that has no gradient yet, for instance."""
    x = CudaLike(torch.zeros(8))
    refused(lambda: clipping.GradClipper([what]), "grads[0] must be a tensor", ar.AR_ERR_INVALID_ARG)
    refused(lambda: clipping.GradClipper([x, what]), "grads[1] must be a tensor", ar.AR_ERR_INVALID_ARG)
    refused(lambda: clipping.GradClipper([x], out=[what]), "out[0] must be a tensor", ar.AR_ERR_INVALID_ARG)
