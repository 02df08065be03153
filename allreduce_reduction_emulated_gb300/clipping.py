"""Global norm of many gradient tensors and clipping by it: what happens to the
gradients between the all-reduce and the update.

    clipper = GradClipper(grads)          # once, like the reducer
    norm = clipper.clip(1.0)              # every step: 0-dim tensor, no host wait

Argument checks and marshalling only; the formulas are in include/ar_train.h.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import (AR_BFLOAT16, AR_ERR_INVALID_ARG, AR_ERR_UNSUPPORTED, AR_FLOAT32, AR_SUCCESS, ArError, _stream_handle,
               library)

_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_capturing = torch.cuda.is_current_stream_capturing
_DTYPES = {torch.float32: (AR_FLOAT32, 4), torch.bfloat16: (AR_BFLOAT16, 2)}  # (code, bytes)


class GradClipper:
    """Norm of, and clipping over, a fixed list of gradient tensors.

    grads   contiguous float32 / bfloat16 CUDA tensors on one device, any sizes and
            alignments; no two may share memory (a tied gradient counts once:
            pass it once)
    out     where the clipped gradients go: tensors of the same sizes and types
            (default: in place)

    The list is checked and its addresses are laid out once; every call reads
    the gradients anew.  The clipper keeps their memory: tensors that are made anew
    (zero_grad(set_to_none=True)) or get another storage need a new clipper, which
    goes best with gradients in flat buffers.  Calls of one clipper share a workspace of 32 KiB: they
    may be on any stream and from any thread but must not overlap on the GPU.  A captured call needs
    its clipper, like its gradients, for as long as it is replayed.
    """

    NORMS = 128   # results handed out of one block; each is written by one call only

    def __init__(self, grads, out=None):
        what = "GradClipper"
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.grads) == 0:
            raise ArError(AR_ERR_INVALID_ARG, f"{what}: no tensors")
        if len(self.out) != len(self.grads):
            raise ArError(AR_ERR_INVALID_ARG, f"{what}: {len(self.grads)} gradients, {len(self.out)} outputs")
        self.device = getattr(self.grads[0], "device", None)
        ats, counts, dtypes = self._laid_out("grads", self.grads)
        outs = ats
        spans = [(at, at + n * size, "grads", i) for i, (at, n, (_, size)) in enumerate(zip(ats, counts, dtypes)) if n]
        if out is not None:
            outs, out_counts, out_dtypes = self._laid_out("out", self.out)
            for i, (at, g, n, m, d, e) in enumerate(zip(outs, ats, out_counts, counts, out_dtypes, dtypes)):
                if n != m or d is not e:
                    raise ArError(AR_ERR_INVALID_ARG, f"{what}: out[{i}] is {n} x {self.out[i].dtype}, the gradient "
                                                      f"is {m} x {self.grads[i].dtype}")
                if n and at != g:
                    spans.append((at, at + n * d[1], "out", i))
        spans.sort()
        for (_, end, a, i), (start, _, b, j) in zip(spans, spans[1:]):
            if start < end:
                raise ArError(AR_ERR_INVALID_ARG, f"{what}: {a}[{i}] and {b}[{j}] share memory")
        n = len(self.grads)
        self._n, self._index = n, self.device.index
        self._memory = [t.untyped_storage() for t in (self.grads if out is None else self.grads + self.out)]
        self._grads = (ctypes.c_void_p * n)(*ats)
        self._outs = (ctypes.c_void_p * n)(*outs)
        self._counts = (ctypes.c_size_t * n)(*counts)
        self._dtypes = (ctypes.c_int * n)(*[code for code, _ in dtypes])
        self._lib = library()
        self._bytes = self._lib.ar_grad_norm_workspace()
        with torch.cuda.device(self.device):
            self._home = torch.cuda.current_stream().cuda_stream
            self._workspace = torch.empty(self._bytes, dtype=torch.uint8, device=self.device)
        self._at = self._workspace.data_ptr()
        self._norms, self._captured = [], []
        # A call's kernels follow one another on the stream, whatever other threads call meanwhile: the library's
        # functions run without the interpreter's lock.
        self._lock = threading.Lock()

    def _laid_out(self, name: str, tensors):
        """(addresses, element counts, _DTYPES entries) of tensors the kernels can walk."""
        what = "GradClipper"
        ats, counts, dtypes = [], [], []
        for i, t in enumerate(tensors):
            if not hasattr(t, "data_ptr"):
                raise ArError(AR_ERR_INVALID_ARG, f"{what}: {name}[{i}] must be a tensor, got {type(t).__name__}")
            kind = _DTYPES.get(t.dtype)
            if kind is None:
                raise ArError(AR_ERR_UNSUPPORTED, f"{what}: {name}[{i}] of {t.dtype}: float32 or bfloat16 needed")
            if not t.is_cuda or not t.is_contiguous():
                raise ArError(AR_ERR_INVALID_ARG, f"{what}: {name}[{i}] is not a contiguous CUDA tensor")
            if t.device != self.device:
                raise ArError(AR_ERR_INVALID_ARG, f"{what}: tensors on {self.device} and {t.device}; "
                                                  "all must be on one GPU")
            ats.append(t.data_ptr())
            counts.append(t.numel())
            dtypes.append(kind)
        return ats, counts, dtypes

    def _begin(self, what: str, stream):
        """(stream handle, a new 0-dim norm): both belong to the call's stream."""
        if _current_device() != self._index:
            raise ArError(AR_ERR_INVALID_ARG, f"{what}: gradients are on {self.device}, the current device is "
                                              f"cuda:{_current_device()}")
        current = torch._C._cuda_getCurrentRawStream(self._index)
        handle = current if stream is None else _stream_handle(stream)
        # The block of norms is memory of the home stream's pool, which is allocated from while home is current.  A
        # captured call has a norm to itself, which the clipper keeps: every replay writes it.
        if handle != self._home or current != self._home or _capturing():
            s = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
            if handle != self._home:
                self._workspace.record_stream(s)
            with torch.cuda.stream(s):
                norm = torch.empty((), dtype=torch.float32, device=self.device)
                if _capturing():
                    self._captured.append(norm)
                return handle, norm
        if not self._norms:
            self._norms.extend(torch.empty(self.NORMS, dtype=torch.float32, device=self.device).unbind())
        return handle, self._norms.pop()

    def norm(self, stream=None):
        """The global norm, a 0-dim float32 tensor."""
        with self._lock:
            handle, norm = self._begin("GradClipper.norm", stream)
            st = self._lib.ar_grad_norm(self._n, self._grads, self._counts, self._dtypes, norm.data_ptr(),
                                        self._at, self._bytes, handle)
        if st != AR_SUCCESS:
            raise ArError(st, "GradClipper.norm")
        return norm

    def clip(self, max_norm: float, eps: float = 1e-6, stream=None):
        """Scales every gradient by min(1, max_norm / (norm + eps)) into `out`;
        returns the norm before clipping, a 0-dim float32 tensor."""
        with self._lock:
            handle, norm = self._begin("GradClipper.clip", stream)
            st = self._lib.ar_clip_grads(self._n, self._grads, self._outs, self._counts, self._dtypes, max_norm, eps,
                                         norm.data_ptr(), self._at, self._bytes, handle)
        if st != AR_SUCCESS:
            raise ArError(st, "GradClipper.clip")
        return norm
