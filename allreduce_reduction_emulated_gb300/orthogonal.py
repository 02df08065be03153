"""Orthogonalised updates of weight matrices by Newton-Schulz products: what the
reduced, clipped gradients become before they are applied.

    ortho = Orthogonalizer(grads, momentum=buffers)     # once, like the clipper
    updates = ortho.update()                             # every step: bf16 matrices
    for w, u in zip(weights, updates): w.sub_(u, alpha=rate)

Argument checks and marshalling only; the formulas are in include/ar_train.h.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import AR_BFLOAT16, AR_ERR_INVALID_ARG, AR_ERR_UNSUPPORTED, AR_FLOAT32, AR_SUCCESS, ArError, library
from .losses import _current_device, _on

_DTYPES = {torch.float32: AR_FLOAT32, torch.bfloat16: AR_BFLOAT16}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


class Orthogonalizer:
    """Momentum and orthogonalisation of a fixed list of gradient matrices.

    grads     contiguous float32 / bfloat16 CUDA tensors on one device, each a matrix
              (rows, cols) or a stack of matrices (..., rows, cols), such as the gradient of an
              expert layer's weights
    out       bfloat16 tensors of the same shapes for the updates (default: made once, and
              written anew by every call); may be the gradients themselves where these are bfloat16
    momentum  float32 tensors of the same shapes, updated by every call: m = beta m + g, and the update is
              made of g + beta m (nesterov) or of m.  None: of the gradients alone
    steps, coefficients, eps    of the Newton-Schulz iteration: X = u / (|u| + eps), then `steps` times
              X <- a X + (b A + c A^2) X with A = X X^T
    scale     factor of the results: a number, a list of one for each tensor, or "shape" for
              sqrt(max(1, rows / cols))

    The list is checked and its addresses are laid out once; every call reads the gradients anew.  The
    object keeps the tensors' memory, and a workspace of a bit more than 4 bytes for each element and 4 for
    each of the smaller sides' squares.  Its calls share both: they may be on any stream and from any thread
    but must not overlap on the GPU, captured ones among them; one on another stream than the object was made on
    waits for what that one had to do then.  A captured call needs its object for as long as it is replayed.
    """

    def __init__(self, grads, out=None, momentum=None, beta: float = 0.95, nesterov: bool = True, steps: int = 5,
                 coefficients=COEFFICIENTS, eps: float = 1e-7, scale=1.0):
        what = "Orthogonalizer"
        self.grads = list(grads)
        if len(self.grads) == 0:
            raise ArError(AR_ERR_INVALID_ARG, f"{what}: no tensors")
        self.device = getattr(self.grads[0], "device", None)
        spans = self._checked("grads", self.grads, tuple(_DTYPES))
        if not isinstance(steps, int) or not 1 <= steps <= 16:
            raise ArError(AR_ERR_INVALID_ARG, f"{what}: steps must be 1 to 16, not {steps!r}")
        coefficients = tuple(coefficients)
        if len(coefficients) != 3:
            raise ArError(AR_ERR_INVALID_ARG, f"{what}: three coefficients needed, got {len(coefficients)}")
        shapes = [tuple(g.shape) for g in self.grads]
        scales = self._scales(scale, shapes)
        if momentum is not None:
            momentum = list(momentum)
            self._alike("momentum", momentum, shapes)
            spans += self._checked("momentum", momentum, (torch.float32,))
        self.momentum = momentum
        if out is not None:
            out = list(out)
            self._alike("out", out, shapes)
            for g, o, span in zip(self.grads, out, self._checked("out", out, (torch.bfloat16,))):
                if not (o.data_ptr() == g.data_ptr() and g.dtype == torch.bfloat16):
                    spans.append(span)
        spans = sorted(s for s in spans if s[0] < s[1])
        for (_, end, a), (start, _, b) in zip(spans, spans[1:]):
            if start < end:
                raise ArError(AR_ERR_INVALID_ARG, f"{what}: {a} and {b} share memory")
        n = len(self.grads)
        self._n, self._index = n, self.device.index
        size = ctypes.c_size_t * n
        counts = []
        for s in shapes:
            k = 1
            for v in s[:-2]:
                k *= v
            counts.append(k)
        self._counts, self._rows, self._cols = size(*counts), size(*[s[-2] for s in shapes]), size(*[s[-1] for s in shapes])
        self._dtypes = (ctypes.c_int * n)(*[_DTYPES[g.dtype] for g in self.grads])
        self._scale = (ctypes.c_float * n)(*scales)
        self._beta, self._nesterov, self._steps, self._eps = float(beta), bool(nesterov), steps, float(eps)
        self._coefficients = (ctypes.c_float * 3)(*coefficients)
        self._lib = library()
        self._bytes = self._lib.ar_orthogonalize_workspace(n, self._counts, self._rows, self._cols, steps)
        if self._bytes == ctypes.c_size_t(-1).value:
            raise ArError(AR_ERR_UNSUPPORTED, f"{what}: sides up to 65536 and stacks up to 4096 matrices")
        with torch.cuda.device(self.device):
            self._home = torch.cuda.current_stream().cuda_stream
            self._workspace = torch.empty(self._bytes, dtype=torch.uint8, device=self.device)
            self.out = [torch.empty(s, dtype=torch.bfloat16, device=self.device) for s in shapes] if out is None else out
            # Kernels on their way on this stream may still use what this memory was before.
            self._free = None if torch.cuda.is_current_stream_capturing() else torch.cuda.current_stream().record_event()
        self._made = out is None
        pointers = ctypes.c_void_p * n
        self._grads = pointers(*[g.data_ptr() for g in self.grads])
        self._outs = pointers(*[o.data_ptr() for o in self.out])
        self._momentum = None if momentum is None else pointers(*[m.data_ptr() for m in momentum])
        self._memory = [t.untyped_storage() for t in self.grads + self.out + (momentum or [])]
        self._lock = threading.Lock()

    def _checked(self, name: str, tensors, dtypes):
        """[(first byte, end, name)] of tensors the kernels can walk."""
        what, spans = "Orthogonalizer", []
        for i, t in enumerate(tensors):
            if not hasattr(t, "data_ptr"):
                raise ArError(AR_ERR_INVALID_ARG, f"{what}: {name}[{i}] must be a tensor, got {type(t).__name__}")
            if t.dtype not in dtypes:
                raise ArError(AR_ERR_UNSUPPORTED, f"{what}: {name}[{i}] of {t.dtype}: "
                                                  f"{' or '.join(str(d)[6:] for d in dtypes)} needed")
            if not t.is_cuda or not t.is_contiguous():
                raise ArError(AR_ERR_INVALID_ARG, f"{what}: {name}[{i}] is not a contiguous CUDA tensor")
            if t.device != self.device:
                raise ArError(AR_ERR_INVALID_ARG, f"{what}: tensors on {self.device} and {t.device}; "
                                                  "all must be on one GPU")
            if t.dim() < 2:
                raise ArError(AR_ERR_INVALID_ARG, f"{what}: {name}[{i}] has {t.dim()} dimensions, matrices needed")
            spans.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), f"{name}[{i}]"))
        return spans

    def _alike(self, name: str, tensors, shapes):
        if len(tensors) != len(shapes):
            raise ArError(AR_ERR_INVALID_ARG, f"Orthogonalizer: {len(shapes)} gradients, {len(tensors)} in {name}")
        for i, (t, s) in enumerate(zip(tensors, shapes)):
            if tuple(getattr(t, "shape", s)) != s:
                raise ArError(AR_ERR_INVALID_ARG, f"Orthogonalizer: {name}[{i}] is {tuple(t.shape)}, the gradient is {s}")

    @staticmethod
    def _scales(scale, shapes):
        if isinstance(scale, str):
            if scale != "shape":
                raise ArError(AR_ERR_INVALID_ARG, f"Orthogonalizer: scale must be numbers or 'shape', not {scale!r}")
            return [max(1.0, s[-2] / max(1, s[-1])) ** 0.5 for s in shapes]
        if isinstance(scale, (int, float)):
            return [float(scale)] * len(shapes)
        scale = [float(v) for v in scale]
        if len(scale) != len(shapes):
            raise ArError(AR_ERR_INVALID_ARG, f"Orthogonalizer: {len(shapes)} gradients, {len(scale)} scales")
        return scale

    def update(self, stream=None):
        """Updates the momentum and writes the orthogonalised updates into `out`, which it returns."""
        what = "Orthogonalizer.update"
        if _current_device() != self._index:
            raise ArError(AR_ERR_INVALID_ARG, f"{what}: gradients are on {self.device}, the current device is "
                                              f"cuda:{_current_device()}")
        with self._lock:
            if stream is None:
                handle = torch._C._cuda_getCurrentRawStream(self._index)
            else:
                handle = _on(stream)[1]
            if handle != self._home:
                s = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
                # (A captured call cannot wait for it, and need not: torch.cuda.graph waits for the GPU before it begins.)
                with torch.cuda.stream(s):
                    if self._free is not None and not torch.cuda.is_current_stream_capturing():
                        s.wait_event(self._free)
                self._workspace.record_stream(s)
                if self._made:
                    for o in self.out:
                        o.record_stream(s)
            st = self._lib.ar_orthogonalize(self._n, self._grads, self._momentum, self._outs, self._counts, self._rows,
                                            self._cols, self._dtypes, self._scale, self._beta, self._nesterov,
                                            self._steps, self._coefficients, self._eps, self._workspace.data_ptr(),
                                            self._bytes, handle)
        if st != AR_SUCCESS:
            raise ArError(st, what)
        return self.out
