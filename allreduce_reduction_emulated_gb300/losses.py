"""Losses over a matrix of logits, with the gradient of the logits: what makes
the gradients that the all-reduce then sums.

    logp = token_logprobs(logits, targets)
    r = policy_loss(logits, targets, old_logprobs, advantages, ref_logprobs=ref, kl_coef=0.05)
    r = preference_loss(logits, targets, offsets, ref_logprobs)
    r.loss, r.grad          # a 0-dim tensor; the gradient of the logits, in their type

Argument checks and marshalling only: the formulas, the treatment of masked
rows (weight 0) and the kernels' contract are in include/ar_train.h.  The
functions build no autograd graph: r.grad is the gradient to send into the
backward pass (logits.backward(r.grad)).

logits        (tokens, vocab) float32 or bfloat16 CUDA tensor on the current
              device; columns contiguous, rows at any stride >= vocab (a view of
              a padded matrix is fine)
targets       (tokens,) int64 or int32
per-token     (tokens,) contiguous float32: weights, old_logprobs, ...
grad          where the gradient goes: a tensor of the logits' shape and type, or
              the logits themselves (in place); None allocates one whose rows start
              at the logits' alignments (for padded or odd layouts it may have a few
              elements between its rows).  A gradient given at other alignments is
              written in narrower stores, which takes longer
stream        a torch stream or a cudaStream_t (default: the current stream).  What is
              allocated belongs to that stream; as with any kernel on a stream of
              one's own, the caller orders it after whatever made the inputs and
              keeps these until the stream is past the call

Nothing waits for the GPU and nothing is kept between calls.
"""
from __future__ import annotations

import torch

from . import AR_BFLOAT16, AR_ERR_INVALID_ARG, AR_ERR_UNSUPPORTED, AR_FLOAT32, AR_SUCCESS, ArError, library

_DTYPES = {torch.float32: AR_FLOAT32, torch.bfloat16: AR_BFLOAT16}
_INDEX_BYTES = {torch.int64: 8, torch.int32: 4}
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _bad(what: str, why: str, status: int = AR_ERR_INVALID_ARG) -> ArError:
    return ArError(status, f"{what}: {why}")


def _matrix(what: str, name: str, x):
    """(device, rows, vocab, row stride) of a matrix the kernels can walk."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise _bad(what, f"{name} must be a 2-dimensional tensor (tokens, vocab)")
    if x.dtype not in _DTYPES:
        raise _bad(what, f"{name} of {x.dtype}: float32 or bfloat16 needed", AR_ERR_UNSUPPORTED)
    device = x.get_device()
    if device < 0:
        raise _bad(what, f"{name} is not in CUDA memory")
    if device != _current_device():
        raise _bad(what, f"{name} is on cuda:{device}, the current device is cuda:{_current_device()}")
    rows, vocab = x.shape
    if rows and not vocab:
        raise _bad(what, f"{name} has no columns")
    stride, column = x.stride()
    if column != 1 and vocab > 1:
        raise _bad(what, f"{name}: columns are not contiguous")
    if rows <= 1:
        stride = vocab
    elif stride < vocab:
        raise _bad(what, f"{name}: rows overlap (stride {stride}, {vocab} columns)")
    return device, rows, vocab, stride


def _vector(what: str, name: str, x, device: int, count: int) -> int:
    """Address of a per-token float32 vector."""
    if not isinstance(x, torch.Tensor):
        raise _bad(what, f"{name} must be a tensor, got {type(x).__name__}")
    if x.dtype != torch.float32:
        raise _bad(what, f"{name} of {x.dtype}: float32 needed", AR_ERR_UNSUPPORTED)
    if x.get_device() != device:
        raise _bad(what, f"{name} is on {x.device}, the logits are on cuda:{device}")
    if x.numel() != count or not x.is_contiguous():
        raise _bad(what, f"{name}: {count} contiguous elements needed, got shape {tuple(x.shape)}")
    return x.data_ptr()


def _indices(what: str, name: str, x, device: int, count: int):
    """(address, bytes per index) of a vector of indices."""
    if not isinstance(x, torch.Tensor):
        raise _bad(what, f"{name} must be a tensor, got {type(x).__name__}")
    size = _INDEX_BYTES.get(x.dtype)
    if size is None:
        raise _bad(what, f"{name} of {x.dtype}: int64 or int32 needed", AR_ERR_UNSUPPORTED)
    if x.get_device() != device:
        raise _bad(what, f"{name} is on {x.device}, the logits are on cuda:{device}")
    if x.numel() != count or not x.is_contiguous():
        raise _bad(what, f"{name}: {count} contiguous elements needed, got shape {tuple(x.shape)}")
    return x.data_ptr(), size


def _gradient(what: str, logits, grad, device: int, rows: int, vocab: int):
    """The tensor for the gradient; None makes one whose rows start at the logits'
    alignments within 16 bytes (then both are read and written in whole vectors)."""
    if grad is None:
        if logits.is_contiguous() and logits.data_ptr() % 16 == 0:
            return torch.empty_like(logits)
        return _like_rows(logits, rows, vocab)
    if grad is not logits:
        at, r, v, stride = _matrix(what, "grad", grad)
        if (at, r, v) != (device, rows, vocab) or grad.dtype != logits.dtype:
            raise _bad(what, f"grad: {tuple(grad.shape)} {grad.dtype}, the logits are {(rows, vocab)} {logits.dtype}")
    return grad


def _like_rows(logits, rows: int, vocab: int):
    """A new matrix whose rows start at the logits' alignments: contiguous, or with
    less than 16 bytes between the rows."""
    size = logits.element_size()
    lead = logits.data_ptr() % 16 // size
    stride = vocab + ((logits.stride(0) - vocab) % (16 // size) if rows > 1 else 0)
    if lead == 0 and stride == vocab:
        return torch.empty((rows, vocab), dtype=logits.dtype, device=logits.device)
    flat = torch.empty(lead + rows * stride, dtype=logits.dtype, device=logits.device)
    return flat.as_strided((rows, vocab), (stride, 1), lead)


def _outputs(what: str, logits, grad, device: int, rows: int, vocab: int, floats: int, stream):
    """(gradient, float buffer, stream handle)"""
    if stream is None:
        return (_gradient(what, logits, grad, device, rows, vocab),
                torch.empty(floats, dtype=torch.float32, device=logits.device),
                torch._C._cuda_getCurrentRawStream(device))
    context, handle = _on(stream)
    with context:
        return (_gradient(what, logits, grad, device, rows, vocab),
                torch.empty(floats, dtype=torch.float32, device=logits.device), handle)


def _on(stream):
    """(the context in which a given stream's outputs are allocated, its handle):
    what is allocated for a stream has to come from that stream's memory pool."""
    if isinstance(stream, int):
        s = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        return torch.cuda.stream(s), stream
    if stream.device_index != _current_device():  # its context would make that device the current one
        raise _bad("stream", f"it is on cuda:{stream.device_index}, the current device is cuda:{_current_device()}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _whole(n: int) -> int:
    """n floats rounded up to whole 16 bytes."""
    return (n + 3) & ~3


def _check(status: int, what: str) -> None:
    if status != AR_SUCCESS:
        raise ArError(status, what)


def token_logprobs(logits, targets, weights=None, out=None, stream=None):
    """Log-probability of each row's target, (tokens,) float32: logits[t, y] -
    logsumexp(logits[t]).  A row of weight 0 is not read and gives 0."""
    what = "token_logprobs"
    device, rows, vocab, stride = _matrix(what, "logits", logits)
    y, size = _indices(what, "targets", targets, device, rows)
    w = None if weights is None else _vector(what, "weights", weights, device, rows)
    if stream is not None:
        context, handle = _on(stream)
        if out is None:
            with context:
                out = torch.empty(rows, dtype=torch.float32, device=logits.device)
    else:
        handle = torch._C._cuda_getCurrentRawStream(device)
        if out is None:
            out = torch.empty(rows, dtype=torch.float32, device=logits.device)
    to = _vector(what, "out", out, device, rows)
    _check(library().ar_token_logprobs(logits.data_ptr(), rows, vocab, stride, _DTYPES[logits.dtype], y, size, w,
                                       to, handle), what)
    return out


class PolicyLoss:
    """What policy_loss computes.  grad is a tensor of its own; loss, kl, clipped and
    weight (0-dim) and logprobs are views of one buffer."""

    __slots__ = ("grad", "_buffer", "_rows")

    def __init__(self, grad, buffer, rows):
        self.grad, self._buffer, self._rows = grad, buffer, rows

    loss = property(lambda self: self._buffer[0], doc="scale * sum of w * term")
    kl = property(lambda self: self._buffer[1], doc="scale * sum of w * (e^d - 1 - d), d = ref - logp")
    clipped = property(lambda self: self._buffer[2], doc="scale * sum of w over the clipped tokens")
    weight = property(lambda self: self._buffer[3], doc="scale * sum of w")
    stats = property(lambda self: self._buffer[:4], doc="loss, kl, clipped, weight")
    logprobs = property(lambda self: self._buffer[4:4 + self._rows], doc="(tokens,) float32, 0 for masked rows")


def policy_loss(logits, targets, old_logprobs, advantages, ref_logprobs=None, weights=None, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, scale: float | None = None, grad=None,
                stream=None) -> PolicyLoss:
    """Clipped policy loss with a KL term to a reference policy, and its gradient.

    loss = scale * sum_t w_t (-min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A)
                              + kl_coef (e^d - 1 - d)),
    r = exp(logp - old), d = ref - logp.  weights=None counts every token; scale=None
    is then 1 / tokens (the mean), and 1 when weights are given (put the
    normalisation into them or into scale: the all-reduce can carry the 1 / P)."""
    what = "policy_loss"
    device, rows, vocab, stride = _matrix(what, "logits", logits)
    y, size = _indices(what, "targets", targets, device, rows)
    w = None if weights is None else _vector(what, "weights", weights, device, rows)
    old = _vector(what, "old_logprobs", old_logprobs, device, rows)
    adv = _vector(what, "advantages", advantages, device, rows)
    ref = None if ref_logprobs is None else _vector(what, "ref_logprobs", ref_logprobs, device, rows)
    if scale is None:
        scale = 1.0 / max(1, rows) if weights is None else 1.0
    lib = library()
    bytes_ = lib.ar_policy_loss_workspace(rows)
    after = 4 + _whole(rows)                       # floats before the workspace: the statistics, logprobs
    grad, buffer, handle = _outputs(what, logits, grad, device, rows, vocab, after + bytes_ // 4, stream)
    at = buffer.data_ptr()
    _check(lib.ar_policy_loss(logits.data_ptr(), rows, vocab, stride, _DTYPES[logits.dtype], y, size, w, old, adv, ref,
                              clip_low, clip_high, kl_coef, scale, grad.data_ptr(),
                              grad.stride(0) if rows > 1 else vocab, at + 16, at, at + 4 * after, bytes_, handle), what)
    return PolicyLoss(grad, buffer, rows)


class PreferenceLoss:
    """What preference_loss computes.  grad is a tensor of its own; loss (0-dim),
    margins and logprobs are views of one buffer."""

    __slots__ = ("grad", "_buffer", "_pairs", "_rows")

    def __init__(self, grad, buffer, pairs, rows):
        self.grad, self._buffer, self._pairs, self._rows = grad, buffer, pairs, rows

    loss = property(lambda self: self._buffer[0])
    margins = property(lambda self: self._buffer[4:4 + self._pairs], doc="(pairs,) float32")

    @property
    def logprobs(self):
        """(tokens,) float32, 0 for masked rows"""
        at = 4 + _whole(self._pairs)
        return self._buffer[at:at + self._rows]


def preference_loss(logits, targets, offsets, ref_logprobs=None, weights=None, beta: float = 0.1,
                    label_smoothing: float = 0.0, scale: float | None = None, grad=None,
                    stream=None) -> PreferenceLoss:
    """Preference loss over pairs of sequences (paired log ratios), and its gradient.

    offsets  (2 * pairs + 1,) int64 or int32 on the GPU: sequence k is rows
             [offsets[k], offsets[k + 1]); sequences 2i and 2i + 1 are the chosen
             and the rejected answer of pair i
    loss = scale * sum_i (1 - label_smoothing) softplus(-z_i) + label_smoothing softplus(z_i),
    z_i = beta * (sum over the chosen rows of w (logp - ref) - the same over the
    rejected).  scale=None is 1 / pairs."""
    what = "preference_loss"
    device, rows, vocab, stride = _matrix(what, "logits", logits)
    y, size = _indices(what, "targets", targets, device, rows)
    w = None if weights is None else _vector(what, "weights", weights, device, rows)
    ref = None if ref_logprobs is None else _vector(what, "ref_logprobs", ref_logprobs, device, rows)
    n = offsets.numel() if isinstance(offsets, torch.Tensor) else 1
    if n % 2 == 0:
        raise _bad(what, f"offsets: 2 * pairs + 1 needed, got {n}")
    off, off_size = _indices(what, "offsets", offsets, device, n)
    pairs = n // 2
    if scale is None:
        scale = 1.0 / max(1, pairs)
    lib = library()
    bytes_ = lib.ar_preference_loss_workspace(rows, pairs)
    first = 4 + _whole(pairs)                      # floats before logprobs: the loss, the margins
    after = first + _whole(rows)
    grad, buffer, handle = _outputs(what, logits, grad, device, rows, vocab, after + bytes_ // 4, stream)
    at = buffer.data_ptr()
    _check(lib.ar_preference_loss(logits.data_ptr(), rows, vocab, stride, _DTYPES[logits.dtype], y, size, w, off,
                                  off_size, pairs, ref, beta, label_smoothing, scale, grad.data_ptr(),
                                  grad.stride(0) if rows > 1 else vocab, at + 4 * first, at, at + 16, at + 4 * after,
                                  bytes_, handle), what)
    return PreferenceLoss(grad, buffer, pairs, rows)
