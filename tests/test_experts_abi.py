"""The expert products and the orthogonalisation without a GPU: the library's argument checks and the
binding's refusals, all before any CUDA call."""
import ctypes
import math

import pytest
import torch

import allreduce_reduction_emulated_gb300 as ar
from allreduce_reduction_emulated_gb300 import _build, experts, losses
from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer
from test_train_abi import BAD, NO, CudaLike, OnGpu, P, refused


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ar.library()


def test_expert_product_arguments(lib):
    def call(x=P, rows=4, x_stride=8, w=P, experts=2, out=16, k=8, es=128, os=8, ks=1, off=P, size=8, y=1 << 20,
             y_stride=16, dtype=ar.AR_BFLOAT16, ws=None, nbytes=0):
        return lib.ar_expert_product(x, rows, x_stride, w, experts, out, k, es, os, ks, off, size, y, y_stride, dtype, 0,
                                     ws, nbytes, None)

    assert call(rows=0) == ar.AR_SUCCESS
    assert call(out=0, os=8, es=0) == ar.AR_SUCCESS
    for kw in (dict(dtype=ar.AR_INT32), dict(rows=(1 << 28) + 1), dict(experts=1025, es=128), dict(out=(1 << 24) + 1),
               dict(k=(1 << 24) + 1, x_stride=1 << 25, os=1 << 25), dict(rows=1 << 28, out=1 << 24, y_stride=1 << 24)):
        assert call(**kw) == NO, kw
    for kw in (dict(dtype=7), dict(x=None), dict(x=P + 1), dict(w=None), dict(w=P + 1), dict(off=None), dict(off=P + 4),
               dict(size=2), dict(y=None), dict(y=(1 << 20) + 1), dict(x_stride=7), dict(y_stride=15), dict(os=7),
               dict(os=2, ks=2), dict(ks=2), dict(es=127), dict(os=1, ks=15), dict(y=P), dict(y=P + 32),
               dict(dtype=ar.AR_FLOAT32, y=(1 << 20) + 2), dict(es=1 << 41), dict(x=P + 2), dict(x_stride=9),
               dict(x=P + 2, ws=P + 8, nbytes=1 << 20)):
        assert call(**kw) == BAD, kw


def test_expert_weight_gradient_arguments(lib):
    def call(dy=P, dys=16, x=P, xs=8, rows=4, experts=2, out=16, k=8, off=P, size=4, dw=1 << 20, es=128, os=8, ks=1,
             dtype=ar.AR_FLOAT32, ws=None, nbytes=0):
        return lib.ar_expert_weight_gradient(dy, dys, x, xs, rows, experts, out, k, off, size, dw, es, os, ks, dtype, 0, ws,
                                             nbytes, None)

    assert call(experts=0) == ar.AR_SUCCESS
    for kw in (dict(dtype=ar.AR_INT32), dict(experts=1025), dict(rows=(1 << 28) + 1)):
        assert call(**kw) == NO, kw
    for kw in (dict(dtype=5), dict(dy=None), dict(dy=P + 1), dict(x=None), dict(dys=15), dict(xs=7), dict(off=None),
               dict(off=P + 2), dict(size=16), dict(dw=None), dict(dw=(1 << 20) + 2), dict(es=127), dict(os=7), dict(ks=3),
               dict(dys=17), dict(xs=12)):
        assert call(**kw) == BAD, kw


def test_expert_workspace(lib):
    f = lib.ar_expert_workspace
    assert f(P, 64, 10, 1, 64, 0) == 0 and f(P, 60, 1, 1, 60, 0) == 0
    assert f(P, 60, 10, 2, 64, 640) == 0
    for at, row, matrix in ((P + 2, 64, 640), (P, 60, 640), (P, 64, 641)):
        assert f(at, 60, 10, 2, row, matrix) >= 10 * 2 * 64 * 2
    assert f(P, 1 << 25, 1, 1, 0, 0) == ctypes.c_size_t(-1).value


def test_expert_parts_workspace(lib):
    f = lib.ar_expert_parts_workspace
    for sizes in ((0, 1, 8, 8), (8, 0, 8, 8), (8, 1, 0, 8), (8, 1, 8, 0)):
        assert f(*sizes, 0) == 0 and f(*sizes, 1) == 0
    for sizes in (((1 << 28) + 1, 1, 8, 8), (8, 1025, 8, 8), (8, 1, (1 << 24) + 1, 8), (8, 1, 8, (1 << 24) + 1)):
        assert f(*sizes, 1) == ctypes.c_size_t(-1).value


def test_orthogonalize_arguments(lib):
    def arrays(kind, values):
        return None if values is None else (kind * len(values))(*values)

    def call(grads=(P, 2 * P), momentum=None, outs=(4 * P, 5 * P), counts=(1, 2), rows=(200, 16), cols=(300, 700),
             dtypes=(0, 1), scales=None, beta=0.95, steps=5, coefs=(3.4445, -4.775, 2.0315), eps=1e-7, ws=P, nbytes=None):
        p, z = ctypes.c_void_p, ctypes.c_size_t
        n, r, c = arrays(z, counts), arrays(z, rows), arrays(z, cols)
        if nbytes is None:
            nbytes = lib.ar_orthogonalize_workspace(len(counts), n, r, c, 5)
        return lib.ar_orthogonalize(len(counts), arrays(p, grads), arrays(p, momentum), arrays(p, outs), n, r, c,
                                    arrays(ctypes.c_int, dtypes), arrays(ctypes.c_float, scales), beta, 1, steps,
                                    arrays(ctypes.c_float, coefs), eps, ws, nbytes, None)

    big = 1 << 40
    for kw in (dict(dtypes=(0, 2)), dict(rows=(1 << 17, 2), nbytes=big), dict(cols=(8, 1 << 17), nbytes=big),
               dict(counts=(1 << 13, 1), nbytes=big)):
        assert call(**kw) == NO, kw
    for kw in (dict(dtypes=(0, 9)), dict(grads=(None, P)), dict(grads=(P + 2, P)), dict(grads=None), dict(outs=(P + 1, P)),
               dict(outs=(None, P)), dict(outs=None), dict(momentum=(P, None)), dict(momentum=(P + 2, P)), dict(steps=0),
               dict(steps=17, nbytes=big), dict(coefs=None), dict(coefs=(math.nan, 0, 0)), dict(coefs=(3.0, math.inf, 0)),
               dict(coefs=(100.0, 0.0, 0.0)), dict(beta=math.nan), dict(eps=-1.0), dict(eps=math.inf),
               dict(scales=(1.0, math.nan)), dict(ws=None), dict(ws=P + 4), dict(nbytes=16)):
        assert call(**kw) == BAD, kw
    one = (ctypes.c_size_t * 1)(1)
    assert lib.ar_orthogonalize_workspace(1, one, one, one, 0) == ctypes.c_size_t(-1).value
    assert lib.ar_orthogonalize_workspace(1, None, one, one, 5) == ctypes.c_size_t(-1).value
    assert call(coefs=(2.0, -1.5, 0.5), counts=(), grads=(), outs=(), rows=(), cols=(), dtypes=(), ws=None) in (
        ar.AR_SUCCESS, ar.AR_ERR_CUDA)


def test_experts_binding_refusals(lib, monkeypatch):
    for m in (losses, experts):
        monkeypatch.setattr(m, "_current_device", lambda: 0)
    g = OnGpu.of
    bf = lambda *s: g(torch.zeros(s, dtype=torch.bfloat16))  # noqa: E731
    x, dy, w, off = bf(6, 8), bf(6, 16), bf(3, 16, 8), g(torch.tensor([0, 2, 4, 6]))
    f, h = experts.expert_product, experts.expert_gradients
    refused(lambda: f(torch.zeros(6, 8, dtype=torch.bfloat16), w, off), "not in CUDA memory")
    refused(lambda: f(None, w, off), "2-dimensional")
    refused(lambda: f(g(torch.zeros(6, 8)), w, off), "bfloat16 needed", NO)
    refused(lambda: f(g(x, 1), w, off), "cuda:1")
    refused(lambda: f(bf(8, 6).t(), w, off), "columns are not contiguous")
    refused(lambda: f(bf(1, 8).expand(6, 8), w, off), "rows overlap")
    refused(lambda: f(x, bf(16, 8), off), "3-dimensional")
    refused(lambda: f(x, g(torch.zeros(3, 16, 8)), off), "bfloat16 needed", NO)
    refused(lambda: f(x, torch.zeros(3, 16, 8, dtype=torch.bfloat16), off), "weights is on")
    refused(lambda: f(x, bf(3, 32, 16)[:, ::2, ::2], off), "contiguous")
    refused(lambda: f(x, bf(1, 16, 8).expand(3, 16, 8), off), "experts overlap")
    refused(lambda: f(x, bf(3, 16, 9), off), "8 columns")
    refused(lambda: f(x, w, g(torch.tensor([0, 6]))), "4 contiguous")
    refused(lambda: f(x, w, g(torch.zeros(4))), "int64 or int32", NO)
    refused(lambda: f(x, w, torch.tensor([0, 2, 4, 6])), "offsets is on cpu")
    refused(lambda: f(x, w, [0, 2, 4, 6]), "offsets must be a tensor")
    refused(lambda: f(x, w, off, dtype=torch.float16), "float32 or bfloat16", NO)
    refused(lambda: f(x, w, off, out=bf(6, 15)), "15 columns")
    refused(lambda: f(x, w, off, out=bf(5, 16)), "5 rows")
    refused(lambda: f(x, w, off, out=g(torch.zeros(6, 16, dtype=torch.float64))), "float32 or bfloat16", NO)
    refused(lambda: f(x, w, off, out=bf(6, 16), dtype=torch.float32), "dtype is")
    refused(lambda: h(bf(5, 16), x, w, off), "6 rows, 5 needed")
    refused(lambda: h(bf(6, 15), x, w, off), "15 columns")
    refused(lambda: h(dy, x, w, off, dx=bf(6, 9)), "dx has 9")
    refused(lambda: h(dy, x, w, off, dw=bf(3, 8, 16)), "dw is")
    refused(lambda: h(dy, x, w, off, dw=bf(3, 16, 8), dw_dtype=torch.float32), "dw_dtype is")
    refused(lambda: h(dy, x, w, off, dw_dtype=torch.int32), "float32 or bfloat16", NO)
    refused(lambda: h(dy, x, w, off, accumulate=True), "accumulate")
    refused(lambda: h(dy, x, w, off, dw=bf(3, 16, 8), accumulate=True, need_dw=False), "accumulate")


def test_orthogonalizer_refusals(lib):
    make = Orthogonalizer
    x = torch.zeros(4, 8)
    c = CudaLike
    refused(lambda: make([]), "no tensors")
    refused(lambda: make([None]), "grads[0] must be a tensor")
    refused(lambda: make([x]), "not a contiguous CUDA tensor")
    refused(lambda: make([c(x.half())]), "float32 or bfloat16", NO)
    refused(lambda: make([c(x.t())]), "not a contiguous CUDA tensor")
    refused(lambda: make([c(x[0])]), "1 dimensions")
    refused(lambda: make([c(x), c(torch.zeros(4, 8), 1)]), "one GPU")
    refused(lambda: make([c(x), c(x)]), "share memory")
    refused(lambda: make([c(x)], momentum=[]), "0 in momentum")
    refused(lambda: make([c(x)], momentum=[c(torch.zeros(8, 4))]), "momentum[0]")
    refused(lambda: make([c(x)], momentum=[c(x)]), "share memory")
    refused(lambda: make([c(x)], momentum=[c(torch.zeros(4, 8, dtype=torch.bfloat16))]), "float32", NO)
    refused(lambda: make([c(x)], out=[c(torch.zeros(4, 8))]), "bfloat16", NO)
    refused(lambda: make([c(x)], out=[c(torch.zeros(4, 9, dtype=torch.bfloat16))]), "out[0]")
    for steps in (0, 17, 2.5):
        refused(lambda: make([c(x)], steps=steps), "steps")
    refused(lambda: make([c(x)], coefficients=(1.0, 2.0)), "three coefficients")
    refused(lambda: make([c(x)], scale="rows"), "'shape'")
    refused(lambda: make([c(x)], scale=[1.0, 2.0]), "2 scales")


def test_results_in_their_inputs(lib, monkeypatch):
    """What a product writes may not be what it reads; columns of one wider matrix are apart."""
    def product(y, y_stride=16, x_stride=8, w=64 * P):
        return lib.ar_expert_product(P, 4, x_stride, w, 2, 16, 8, 128, 8, 1, P, 8, y, y_stride, ar.AR_BFLOAT16, 0, None, 0,
                                     None)

    def gradient(dw, dtype=ar.AR_BFLOAT16):
        return lib.ar_expert_weight_gradient(64 * P, 16, P, 8, 4, 2, 16, 8, P, 8, dw, 128, 8, 1, dtype, 0, None, 0, None)

    launched = (ar.AR_SUCCESS, ar.AR_ERR_CUDA)  # what a call answers that is not refused, without a GPU
    if torch.cuda.is_available():
        pytest.skip("the addresses are stand-ins")
    # the weights span (128 + 15 * 8 + 8) * 2 bytes, y 4 * 16 * 2
    for y in (64 * P, 64 * P + 510, 64 * P - 126, P, P + 62, P - 126):
        assert product(y) == BAD, y
    for y in (64 * P + 512, 64 * P - 128, P + 64, P - 128):
        assert product(y) in launched, y
    # x in the first 8 of 24 columns, y in the others; then one column too far to the left, or too wide a row
    assert product(P + 16, 24, 24) in launched and product(P + 16 + 48, 24, 24) in launched
    assert product(P - 32, 24, 24) in launched
    for y, stride in ((P + 14, 24), (P + 16, 23), (P - 30, 24), (P + 18, 24)):
        assert product(y, stride, 24) == BAD, (y, stride)
    for dw in (P, P + 62, P - 510, 64 * P, 64 * P + 126, 64 * P - 510):
        assert gradient(dw) == BAD, dw
    assert gradient(P - 1022 + 2, ar.AR_FLOAT32) == BAD
    for dw in (P + 64, P - 512, 64 * P + 128, 64 * P - 512):
        assert gradient(dw) in launched, dw

    for m in (losses, experts):
        monkeypatch.setattr(m, "_current_device", lambda: 0)
    g, h = OnGpu.of, experts.expert_gradients
    both = torch.zeros(6, 24, dtype=torch.bfloat16)
    x, dy, w = g(both[:, :8]), g(torch.zeros(6, 16, dtype=torch.bfloat16)), g(torch.zeros(3, 16, 8, dtype=torch.bfloat16))
    off = g(torch.tensor([0, 2, 4, 6]))
    refused(lambda: h(dy, x, w, off, dx=x), "dx and x share")
    refused(lambda: h(dy, x, w, off, dx=g(both[:, 7:15])), "dx and x share")
    refused(lambda: h(dy, x, w, off, dx=g(both.view(-1)[3:99].view(6, 16)[:, :8])), "dx and x share")
    flat = torch.zeros(3 * 16 * 8, dtype=torch.bfloat16)
    refused(lambda: h(dy, x, w, off, dx=g(flat[336:].view(6, 8)), dw=g(flat.view(3, 16, 8))), "dx and dw share")
    assert not experts._shared(both[:, :8], both[:, 8:]) and not experts._shared(both[:, 8:], both[:, :8])
    assert experts._shared(both[:, :9], both[:, 8:]) and experts._shared(both[:, 20:], both[1:, :3]) is False
