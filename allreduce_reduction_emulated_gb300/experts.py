"""Products of rows sorted by expert with their expert's weights, and their
gradients: the layers between the logits' gradient and the weights' gradients.

    y = expert_product(x, weights, offsets)
    dx, dw = expert_gradients(dy, x, weights, offsets)

Argument checks and marshalling only: the formulas and the kernels' contract are in
include/ar_train.h.  The functions build no autograd graph.

x, dy         (rows, in) and (rows, out) bfloat16 CUDA tensors on the current device;
              columns contiguous, rows at any stride
weights       (experts, out, in) bfloat16; `in` or `out` contiguous, the other two at
              any strides (a transposed view is fine)
offsets       (experts + 1,) int64 or int32 on the GPU: expert e has rows
              [offsets[e], offsets[e + 1]).  Nothing waits for their values
stream        a torch stream or a cudaStream_t (default: the current stream).  What is
              allocated belongs to that stream

Rows of no expert (in front of offsets[0], behind offsets[-1]) are left as they are in
a result that is given, and 0 in one that the call makes.  Operands whose address or
strides are not whole 16 bytes are copied to a workspace first, which takes longer.
bfloat16 results of sums over more than 2^18 products go by way of float32 ones.
Nothing waits for the GPU and nothing is kept between calls.
"""
from __future__ import annotations

import torch

from . import AR_BFLOAT16, AR_ERR_UNSUPPORTED, AR_FLOAT32, library
from .losses import _bad, _check, _current_device, _indices, _on

_DTYPES = {torch.float32: AR_FLOAT32, torch.bfloat16: AR_BFLOAT16}

# The tensor cores cut what an addition loses, on average 2^-25 of the sum for every 16 products: over so many it is an
# eighth of bfloat16's half step.  Longer sums of a bfloat16 result are made in float32, which adds them up in runs.
_LONGEST = 1 << 18

# More bytes than any workspace of sizes within the limits that fits a GPU.
_LARGEST = 1 << 48

# Shorter sums, or more tiles of 128 x 128, are never split into parts: no call to ask.
_LONG, _FEW = 1024, 256


def _rows(what: str, name: str, x, device: int | None = None, rows: int | None = None, dtypes=(torch.bfloat16,)):
    """(device, rows, columns, row stride) of a matrix that the kernels can walk."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise _bad(what, f"{name} must be a 2-dimensional tensor (rows, columns)")
    if x.dtype not in dtypes:
        raise _bad(what, f"{name} of {x.dtype}: {' or '.join(str(d)[6:] for d in dtypes)} needed", AR_ERR_UNSUPPORTED)
    at = x.get_device()
    if at < 0:
        raise _bad(what, f"{name} is not in CUDA memory")
    if device is None:
        if at != _current_device():
            raise _bad(what, f"{name} is on cuda:{at}, the current device is cuda:{_current_device()}")
    elif at != device:
        raise _bad(what, f"{name} is on {x.device}, the other tensors are on cuda:{device}")
    n, columns = x.shape
    if rows is not None and n != rows:
        raise _bad(what, f"{name} has {n} rows, {rows} needed")
    stride, column = x.stride()
    if column != 1 and columns > 1:
        raise _bad(what, f"{name}: columns are not contiguous")
    if n <= 1:
        stride = columns
    elif stride < columns:
        raise _bad(what, f"{name}: rows overlap (stride {stride}, {columns} columns)")
    return at, n, columns, stride


def _weights(what: str, name: str, w, device: int, dtypes=(torch.bfloat16,)):
    """(experts, out, in, expert stride, out stride, in stride)"""
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise _bad(what, f"{name} must be a 3-dimensional tensor (experts, out, in)")
    if w.dtype not in dtypes:
        raise _bad(what, f"{name} of {w.dtype}: {' or '.join(str(d)[6:] for d in dtypes)} needed", AR_ERR_UNSUPPORTED)
    if w.get_device() != device:
        raise _bad(what, f"{name} is on {w.device}, the other tensors are on cuda:{device}")
    E, N, K = w.shape
    e, n, k = w.stride()
    # a side of length one has no stride of its own
    if K == 1 and n == 1 and N > 1:
        k = N
    elif K == 1:
        k = 1
        n = max(n, 1) if N > 1 else 1
    elif N == 1:
        n = K if k == 1 else 1
    if not ((k == 1 and n >= K) or (n == 1 and k >= N)) and w.numel():
        raise _bad(what, f"{name}: `in` or `out` must be contiguous and rows must not overlap, got strides {w.stride()}")
    whole = (N - 1) * n + (K - 1) * k + 1
    if E > 1 and e < whole and w.numel():
        raise _bad(what, f"{name}: experts overlap (stride {e}, a matrix spans {whole})")
    return E, N, K, e, n, k


def _shared(a, b) -> bool:
    """Whether two tensors share memory.  Columns of one wider matrix do not."""
    def span(t):
        return sum((n - 1) * s for n, s in zip(t.shape, t.stride())) * t.element_size() + t.element_size()

    if not a.numel() or not b.numel():
        return False
    if b.data_ptr() < a.data_ptr():
        a, b = b, a
    way = b.data_ptr() - a.data_ptr()
    if way >= span(a):
        return False
    row = a.stride(0) * a.element_size()
    if a.dim() == b.dim() == 2 and len(a) > 1 and row == b.stride(0) * b.element_size():
        return way % row < a.shape[1] * a.element_size() or way % row + b.shape[1] * b.element_size() > row
    return True


def _space(lib, device, parts, *operands) -> tuple:
    """(tensor or None, address, bytes) of the workspace of (address, columns, rows, count, row stride, matrix
    stride) operands; none where all of them are aligned, which needs no call to know.  parts: bytes more."""
    bits = 0
    for at, _, _, _, row, matrix in operands:
        bits |= at | row << 1 | matrix << 1
    n = parts + sum(lib.ar_expert_workspace(*o) for o in operands) if bits & 15 else parts
    if not n or n > _LARGEST:   # (of sizes beyond the limits, which the library's call refuses)
        return None, None, 0
    t = torch.empty(n, dtype=torch.uint8, device=device)
    return t, t.data_ptr(), n


def _product(what, lib, x, at_x, w, at_w, offsets, off_size, out, zero_rest, handle):
    """y = the product into `out`; at_w: (experts, out, in, strides)."""
    _, rows, K, x_stride = at_x
    E, N, _, e, n, k = at_w
    x_at, w_at = x.data_ptr(), w.data_ptr()
    by_weights = (w_at, K, N, E, n, e) if k == 1 else (w_at, N, K, E, k, e)
    parts = 0
    if K >= _LONG and -(-N // 128) * (min(E, rows) + rows // 128) <= _FEW:
        parts = lib.ar_expert_parts_workspace(rows, E, N, K, 0)
    space, at, bytes_ = _space(lib, x.device, parts, (x_at, K, rows, 1, x_stride, 0), by_weights)
    _check(lib.ar_expert_product(x_at, rows, x_stride, w_at, E, N, K, e, n, k, offsets, off_size, out.data_ptr(),
                                 out.stride(0) if rows > 1 else N, _DTYPES[out.dtype], zero_rest, at, bytes_, handle),
           what)


def _of(x, shape, dtype):
    """A new tensor beside x."""
    return torch.empty(shape, dtype=dtype, device=x.device)


def _rounded(what, lib, x, at_x, w, at_w, offsets, off_size, out, fresh, handle):
    """_product, by way of float32 where its sums are too long to be rounded once."""
    if at_x[2] <= _LONGEST or out.dtype == torch.float32:
        return _product(what, lib, x, at_x, w, at_w, offsets, off_size, out, fresh, handle)
    if not fresh and (_shared(out, x) or _shared(out, w)):  # which the library cannot see
        raise _bad(what, "the result shares memory with what it is made of")
    wide = _of(x, out.shape, torch.float32) if fresh else out.float()
    _product(what, lib, x, at_x, w, at_w, offsets, off_size, wide, fresh, handle)
    out.copy_(wide)


def expert_product(x, weights, offsets, out=None, dtype=None, stream=None):
    """y[t] = weights[e] @ x[t] for the rows t of each expert e: (rows, out).

    dtype   of a result that the call makes: bfloat16 (default) or float32
    out     where the result goes: (rows, out), bfloat16 or float32, rows at any stride"""
    what = "expert_product"
    at_x = device, rows, K, _ = _rows(what, "x", x)
    at_w = _weights(what, "weights", weights, device)
    E, N = at_w[:2]
    if at_w[2] != K:
        raise _bad(what, f"x has {K} columns, the weights take {at_w[2]}")
    off, size = _indices(what, "offsets", offsets, device, E + 1)
    if out is None:
        if dtype is not None and dtype not in _DTYPES:
            raise _bad(what, f"dtype {dtype}: float32 or bfloat16 needed", AR_ERR_UNSUPPORTED)
    else:
        if _rows(what, "out", out, device, rows, tuple(_DTYPES))[2] != N:
            raise _bad(what, f"out has {out.shape[1]} columns, {N} needed")
        if dtype is not None and out.dtype != dtype:
            raise _bad(what, f"out is {out.dtype}, dtype is {dtype}")
    if stream is not None:
        context, handle = _on(stream)
        with context:
            return _into(what, x, at_x, weights, at_w, off, size, out, dtype, handle)
    return _into(what, x, at_x, weights, at_w, off, size, out, dtype, torch._C._cuda_getCurrentRawStream(device))


def _into(what, x, at_x, weights, at_w, off, size, out, dtype, handle):
    fresh = out is None
    if fresh:
        out = _of(x, (at_x[1], at_w[1]), torch.bfloat16 if dtype is None else dtype)
    _rounded(what, library(), x, at_x, weights, at_w, off, size, out, fresh, handle)
    return out


def expert_gradients(dy, x, weights, offsets, dx=None, dw=None, dw_dtype=None, accumulate: bool = False, need_dx=True,
                     need_dw=True, stream=None):
    """(dx, dw): the gradients of expert_product's x and weights from that of its result.

    dx[t] = weights[e]^T dy[t];  dw[e] = sum over e's rows of dy[t] x[t]^T

    dx, dw      where they go; None makes dx in bfloat16 and dw in dw_dtype (bfloat16
                by default, or float32), laid out as the weights are.  A given dw may be a view
                of a flat gradient buffer.  None of it may be part of an input
    accumulate  add to the dw that is given (an expert without rows keeps its own)
    need_dx, need_dw   False leaves one out (None in its place)"""
    what = "expert_gradients"
    at_y = device, rows, N, dy_stride = _rows(what, "dy", dy)
    at_x = _rows(what, "x", x, device, rows)
    K, x_stride = at_x[2:]
    at_w = _weights(what, "weights", weights, device)
    E = at_w[0]
    if at_w[1:3] != (N, K):
        raise _bad(what, f"dy has {N} columns and x {K}, the weights are {tuple(at_w[1:3])}")
    off, size = _indices(what, "offsets", offsets, device, E + 1)
    if accumulate and (dw is None or not need_dw):
        raise _bad(what, "accumulate needs a dw to add to")
    if dx is not None and need_dx and _rows(what, "dx", dx, device, rows, tuple(_DTYPES))[2] != K:
        raise _bad(what, f"dx has {dx.shape[1]} columns, {K} needed")
    at_dw = None
    if dw is not None and need_dw:
        at_dw = _weights(what, "dw", dw, device, tuple(_DTYPES))
        if at_dw[:3] != (E, N, K):
            raise _bad(what, f"dw is {tuple(dw.shape)}, the weights are {(E, N, K)}")
        if dw_dtype is not None and dw.dtype != dw_dtype:
            raise _bad(what, f"dw is {dw.dtype}, dw_dtype is {dw_dtype}")
    elif dw_dtype is not None and dw_dtype not in _DTYPES:
        raise _bad(what, f"dw_dtype {dw_dtype}: float32 or bfloat16 needed", AR_ERR_UNSUPPORTED)
    if not need_dx:
        dx = None
    if not need_dw:
        dw = None
    if dx is not None and need_dw:  # dx is written before x is read again
        for name, t in ("x", x), ("dw", dw):
            if t is not None and _shared(dx, t):
                raise _bad(what, f"dx and {name} share memory")
    if at_dw is not None and rows and dw.numel():  # before dx is launched
        e, n, k = at_dw[3:]
        begin = dw.data_ptr()
        end = begin + ((E - 1) * e + (N - 1) * n + (K - 1) * k + 1) * dw.element_size()
        for name, t, (_, _, columns, row) in ("x", x, at_x), ("dy", dy, at_y):
            at = t.data_ptr()
            if at < end and begin < at + ((rows - 1) * row + columns) * 2:
                raise _bad(what, f"dw and {name} share memory")
    if stream is not None:
        context, handle = _on(stream)
        with context:
            return _both(what, dy, at_y, x, at_x, weights, at_w, off, size, dx, dw, at_dw, dw_dtype, accumulate, need_dx,
                         need_dw, handle)
    return _both(what, dy, at_y, x, at_x, weights, at_w, off, size, dx, dw, at_dw, dw_dtype, accumulate, need_dx, need_dw,
                 torch._C._cuda_getCurrentRawStream(device))


def _both(what, dy, at_y, x, at_x, weights, at_w, off, size, dx, dw, at_dw, dw_dtype, accumulate, need_dx, need_dw,
          handle):
    lib = library()
    E, N, K, e, n, k = at_w
    _, rows, _, dy_stride = at_y
    x_stride = at_x[3]
    if need_dx:
        fresh = dx is None
        if fresh:
            dx = _of(x, (rows, K), torch.bfloat16)
        _rounded(what, lib, dy, at_y, weights, (E, K, N, e, k, n), off, size, dx, fresh, handle)
    if need_dw:
        def new(dtype):
            if k == 1:
                return _of(x, (E, N, K), dtype), (E, N, K, N * K, K, 1)
            return _of(x, (E, K, N), dtype).transpose(1, 2), (E, N, K, N * K, 1, N)

        if dw is None:
            dw, at_dw = new(torch.bfloat16 if dw_dtype is None else dw_dtype)
        to = dw
        if rows > _LONGEST and dw.dtype == torch.bfloat16:
            to, at_dw = new(torch.float32)
            if accumulate:
                to.copy_(dw)
        dy_at, x_at = dy.data_ptr(), x.data_ptr()
        parts = 0
        if rows >= _LONG * E and -(-N // 128) * -(-K // 128) * E <= _FEW:
            parts = lib.ar_expert_parts_workspace(rows, E, N, K, 1)
        space, at, bytes_ = _space(lib, x.device, parts, (dy_at, N, rows, 1, dy_stride, 0),
                                   (x_at, K, rows, 1, x_stride, 0))
        _check(lib.ar_expert_weight_gradient(dy_at, dy_stride, x_at, x_stride, rows, E, N, K, off, size, to.data_ptr(),
                                             *at_dw[3:], _DTYPES[to.dtype], accumulate, at, bytes_, handle), what)
        if to is not dw:
            dw.copy_(to)
    return dx, dw
