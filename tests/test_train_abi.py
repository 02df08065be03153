"""The training operators without a GPU: the library's argument checks and the
binding's refusals, all before any CUDA call."""
import ctypes
import math

import pytest
import torch

import allreduce_reduction_emulated_gb300 as ar
from allreduce_reduction_emulated_gb300 import _build, clipping, losses

BAD, NO = ar.AR_ERR_INVALID_ARG, ar.AR_ERR_UNSUPPORTED
P = 4096       # stands for a device address; nothing is launched


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ar.library()


def test_token_logprobs_arguments(lib):
    def call(logits=P, rows=4, vocab=8, stride=8, dtype=ar.AR_FLOAT32, targets=P, size=8, weights=None, out=P):
        return lib.ar_token_logprobs(logits, rows, vocab, stride, dtype, targets, size, weights, out, None)

    assert call(rows=0) == ar.AR_SUCCESS
    for kw in (dict(dtype=ar.AR_INT32), dict(rows=(1 << 28) + 1), dict(vocab=(1 << 30) + 1, stride=1 << 31)):
        assert call(**kw) == NO, kw
    for kw in (dict(dtype=7), dict(logits=None), dict(logits=P + 2), dict(vocab=0), dict(stride=7), dict(targets=None),
               dict(targets=P + 4), dict(size=2), dict(out=None), dict(out=P + 1), dict(weights=P + 3),
               dict(rows=1 << 28, stride=1 << 40), dict(dtype=ar.AR_BFLOAT16, logits=P + 1)):
        assert call(**kw) == BAD, kw


def test_policy_loss_arguments(lib):
    need = lib.ar_policy_loss_workspace(4)
    assert need > 0
    assert lib.ar_policy_loss_workspace(1 << 60) == ctypes.c_size_t(-1).value

    def call(logits=P, rows=4, vocab=8, stride=8, dtype=ar.AR_FLOAT32, targets=P, size=8, weights=None, old=P, adv=P,
             ref=None, lo=0.2, hi=0.2, kl=0.0, scale=1.0, grad=1 << 20, gstride=8, lp=P, stats=P, ws=P, nbytes=need):
        return lib.ar_policy_loss(logits, rows, vocab, stride, dtype, targets, size, weights, old, adv, ref, lo, hi, kl,
                                  scale, grad, gstride, lp, stats, ws, nbytes, None)

    assert call(dtype=ar.AR_INT32) == NO
    for kw in (dict(old=None), dict(adv=P + 1), dict(ref=P + 2), dict(lo=-0.1), dict(hi=math.nan), dict(kl=math.nan),
               dict(scale=math.nan), dict(grad=None), dict(gstride=7), dict(stats=None), dict(ws=None),
               dict(ws=P + 8), dict(nbytes=need - 1), dict(lp=None),
               dict(grad=P + 32), dict(grad=P, gstride=9), dict(grad=P - 4)):
        assert call(**kw) == BAD, kw


def test_preference_loss_arguments(lib):
    need = lib.ar_preference_loss_workspace(4, 2)
    assert need >= 4 * 8 + 2 * 12
    assert lib.ar_preference_loss_workspace(1 << 60, 1) == ctypes.c_size_t(-1).value

    def call(rows=4, dtype=ar.AR_FLOAT32, off=P, off_size=8, pairs=2, ref=None, beta=0.1, ls=0.0, scale=1.0,
             grad=1 << 20, loss=P, margins=P, ws=P, nbytes=need):
        return lib.ar_preference_loss(P, rows, 8, 8, dtype, P, 8, None, off, off_size, pairs, ref, beta, ls, scale,
                                      grad, 8, P, loss, margins, ws, nbytes, None)

    assert call(dtype=ar.AR_INT32) == NO
    for kw in (dict(off=None), dict(off=P + 4), dict(off_size=3), dict(ref=P + 2), dict(beta=math.nan), dict(ls=-0.1),
               dict(ls=1.1), dict(ls=math.nan), dict(scale=math.nan), dict(loss=None), dict(margins=None),
               dict(ws=None), dict(nbytes=need - 1), dict(grad=P + 4)):
        assert call(**kw) == BAD, kw


def test_grads_arguments(lib):
    need = lib.ar_grad_norm_workspace()

    def call(ptrs=(P, 2 * P), counts=(4, 4), dtypes=(0, 1), outs=None, max_norm=1.0, eps=1e-6, norm=P, ws=P,
             nbytes=need):
        n = len(ptrs)
        arr = (ctypes.c_void_p * n)(*ptrs)
        out = None if outs is None else (ctypes.c_void_p * n)(*outs)
        sizes, types = (ctypes.c_size_t * n)(*counts), (ctypes.c_int * n)(*dtypes)
        got = lib.ar_clip_grads(n, arr, out, sizes, types, max_norm, eps, norm, ws, nbytes, None)
        if outs is None and max_norm == 1.0 and eps == 1e-6:
            assert got == lib.ar_grad_norm(n, arr, sizes, types, norm, ws, nbytes, None)
        return got

    assert call(dtypes=(0, 2)) == NO
    for kw in (dict(dtypes=(0, 9)), dict(ptrs=(None, P)), dict(ptrs=(P + 2, P)), dict(ptrs=(P, P + 1)),
               dict(counts=(1 << 62, 1)), dict(outs=(P + 4, 2 * P)), dict(outs=(None, 2 * P)), dict(max_norm=-1.0),
               dict(max_norm=math.nan), dict(eps=-1.0), dict(eps=math.nan), dict(norm=None), dict(ws=None),
               dict(ws=P + 4), dict(nbytes=need - 1)):
        assert call(**kw) == BAD, kw
    assert lib.ar_grad_norm(2, None, None, None, P, P, need, None) == BAD


def refused(call, reason, status=BAD):
    with pytest.raises(ar.ArError) as e:
        call()
    assert e.value.status == status and reason in str(e.value), str(e.value)


def test_binding_refuses_what_is_not_a_cuda_matrix(lib):
    x, y, v = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    off = torch.tensor([0, 2, 4])
    for f in (lambda x: losses.token_logprobs(x, y), lambda x: losses.policy_loss(x, y, v, v),
              lambda x: losses.preference_loss(x, y, off)):
        refused(lambda: f(x), "not in CUDA memory")
        refused(lambda: f(x[0]), "2-dimensional")
        refused(lambda: f(None), "2-dimensional")
        refused(lambda: f(x.half()), "float32 or bfloat16", NO)
        refused(lambda: f(x.double()), "float32 or bfloat16", NO)


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on a GPU: for the checks that come after."""

    index = 0

    @staticmethod
    def of(t, index=0):
        t = t.as_subclass(OnGpu)
        t.index = index
        return t

    def get_device(self):
        return self.index


def test_binding_checks_layouts(lib, monkeypatch):
    monkeypatch.setattr(losses, "_current_device", lambda: 0)
    g = OnGpu.of
    x, y, v = g(torch.zeros(4, 8)), g(torch.zeros(4, dtype=torch.int64)), g(torch.zeros(4))
    off = g(torch.tensor([0, 2, 4]))
    f = losses.policy_loss
    refused(lambda: f(g(torch.zeros(4, 8), 1), y, v, v), "cuda:1")
    refused(lambda: f(g(torch.zeros(8, 4).t()), y, v, v), "columns are not contiguous")
    refused(lambda: f(g(torch.zeros(1, 8).expand(4, 8)), y, v, v), "rows overlap")
    refused(lambda: f(g(torch.zeros(4, 0)), y, v, v), "no columns")
    refused(lambda: f(x, g(torch.zeros(3, dtype=torch.int64)), v, v), "4 contiguous")
    refused(lambda: f(x, g(torch.zeros(4)), v, v), "int64 or int32", NO)
    refused(lambda: f(x, torch.zeros(4, dtype=torch.int64), v, v), "targets is on cpu")
    refused(lambda: f(x, y, g(torch.zeros(5)), v), "old_logprobs")
    refused(lambda: f(x, y, v, g(torch.zeros(8)[::2])), "advantages")
    refused(lambda: f(x, y, v, v, g(torch.zeros(4, dtype=torch.float64))), "ref_logprobs", NO)
    refused(lambda: f(x, y, v, v, weights=torch.zeros(4)), "weights is on cpu")
    refused(lambda: losses.preference_loss(x, y, g(torch.tensor([0, 4]))), "2 * pairs + 1")
    refused(lambda: losses.preference_loss(x, y, torch.tensor([0, 2, 4])), "offsets is on cpu")
    refused(lambda: losses.preference_loss(x, y, g(torch.zeros(3))), "int64 or int32", NO)
    for grad in (torch.zeros(4, 9), torch.zeros(3, 8), torch.zeros(4, 8, dtype=torch.bfloat16)):
        refused(lambda: losses._gradient("x", x, g(grad), 0, 4, 8), "grad")
    assert losses._gradient("x", x, x, 0, 4, 8) is x


def test_binding_refuses_what_is_not_a_tensor(lib, monkeypatch):
    monkeypatch.setattr(losses, "_current_device", lambda: 0)
    g = OnGpu.of
    x, y, v = g(torch.zeros(4, 8)), g(torch.zeros(4, dtype=torch.int64)), g(torch.zeros(4))
    refused(lambda: losses.token_logprobs(x, None), "targets must be a tensor")
    refused(lambda: losses.token_logprobs(x, [0, 1, 2, 3]), "targets must be a tensor")
    refused(lambda: losses.policy_loss(x, y, None, v), "old_logprobs must be a tensor")
    refused(lambda: losses.policy_loss(x, y, v, 1.0), "advantages must be a tensor")
    refused(lambda: losses.policy_loss(x, y, v, v, weights=[1.0] * 4), "weights must be a tensor")
    refused(lambda: losses.preference_loss(x, y, [0, 2, 4]), "offsets must be a tensor")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,pad,shift", [(24, 0, 1), (24, 8, 0), (24, 5, 0), (25, 3, 2), (9, 40, 7), (1, 1, 0)])
def test_a_new_gradient_has_the_logits_alignments(dtype, vocab, pad, shift):
    whole = torch.zeros(6, vocab + pad + shift, dtype=dtype)
    x = whole[:, shift:shift + vocab]
    g = losses._like_rows(x, 6, vocab)
    assert g.shape == x.shape and g.dtype == dtype and g.stride(1) == 1 and vocab <= g.stride(0) < vocab + 8
    for t in range(6):
        assert (g[t].data_ptr() - x[t].data_ptr()) % 16 == 0


class CudaLike:
    """A stand-in for a CUDA tensor (a CPU tensor's memory)."""

    def __init__(self, t, index=0):
        self.t, self.is_cuda, self.dtype, self.device = t, True, t.dtype, torch.device("cuda", index)

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_clipper_refusals(lib):
    make = clipping.GradClipper
    x = torch.zeros(16)
    refused(lambda: make([]), "no tensors")
    refused(lambda: make([x]), "not a contiguous CUDA tensor")
    refused(lambda: make([x.half()]), "float32 or bfloat16", NO)
    refused(lambda: make([CudaLike(x[::2])]), "not a contiguous CUDA tensor")
    refused(lambda: make([CudaLike(x[:8]), CudaLike(torch.zeros(4), 1)]), "one GPU")
    refused(lambda: make([CudaLike(x[:8]), CudaLike(x[7:])]), "share memory")
    refused(lambda: make([CudaLike(x), CudaLike(x)]), "share memory")
    refused(lambda: make([CudaLike(x[:8])], out=[]), "0 outputs")
    refused(lambda: make([CudaLike(x[:8])], out=[CudaLike(torch.zeros(9))]), "out[0]")
    refused(lambda: make([CudaLike(x[:8])], out=[CudaLike(x[4:12])]), "share memory")
    refused(lambda: make([CudaLike(x[:4]), CudaLike(x[4:8])], out=[CudaLike(x[4:8]), CudaLike(x[:4])]), "share memory")
    refused(lambda: make([CudaLike(x[:8])], out=[CudaLike(torch.zeros(8, dtype=torch.bfloat16))]), "out[0]")
