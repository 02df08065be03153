"""Plain 64-bit forms of the training operators, and tolerances, for their tests.

Tolerances (fp32 statistics): with z = x - max, e^z carries a relative error of
at most |z| 2^-23 (the difference and its product with log2 e are rounded) plus
2^-22 (the instruction); terms that matter to the sum have |z| < 16, and a
thread adds at most about 600 of them (relative 2^-24 each, in random
directions: under 2e-6).  So log S is within 4e-6, and lp = (x_y - m) - log S
within 4e-6 + 2^-22 |lp|.  The gradient c ([j == y] - p_j) has p within
4e-6 + 2^-23 |z| of its value (|z| <= 40 where p matters: 2e-5 covers both and
the error of c, which is that of e^(lp - old)), the target's 1 - p within p
times lp's error, and one rounding to bf16 (2^-9) where the type is bf16.
"""
import math

import torch

LP_ABS, LP_REL = 4e-6, 2.0 ** -22


def rows64(logits, targets, weights=None):
    """(lp, p) in 64 bits; masked rows give lp 0 and p 0 whatever they hold."""
    x = logits.double()
    if weights is not None:
        x = torch.where((weights != 0)[:, None], x, 0.0)
    logp = torch.log_softmax(x, 1)
    y = targets.long().clamp(0, max(0, x.shape[1] - 1))
    lp = logp.gather(1, y[:, None]).squeeze(1) if len(x) else x.new_zeros(0)
    p = logp.exp()
    if weights is not None:
        lp, p = torch.where(weights != 0, lp, 0.0), torch.where((weights != 0)[:, None], p, 0.0)
    return lp, p


def policy64(logits, targets, old, adv, ref, w, lo=0.2, hi=0.2, kl_coef=0.0, scale=1.0, lp=None):
    """loss, kl, clipped, weight, lp, c (the row factors) and p; with `lp` given, from it."""
    p = None
    if lp is None:
        lp, p = rows64(logits, targets, w)
    on = w != 0
    w64 = torch.where(on, w.double(), 0.0)
    z = lambda v: torch.where(on, v.double(), 0.0)  # noqa: E731
    A, u = z(adv), lp - z(old)
    r = u.exp()
    clipped = on & (((A > 0) & (r > 1 + hi)) | ((A < 0) & (r < 1 - lo)))
    term = -torch.minimum(r * A, r.clamp(1 - lo, 1 + hi) * A)
    d = torch.where(clipped, 0.0, -A * r)
    size = A.abs() * r
    kl = torch.zeros_like(r)
    if ref is not None:
        q = z(ref) - lp
        kl = torch.expm1(q) - q
        term = term + kl_coef * kl
        d = d - kl_coef * torch.expm1(q)
        size = size + kl_coef * (1 + q.exp())
    return {"loss": scale * (w64 * term).sum(), "kl": scale * (w64 * kl).sum(),
            "clipped": scale * (w64 * clipped).sum(), "weight": scale * w64.sum(), "logprobs": lp,
            "c": scale * w64 * d, "size": (scale * w64 * size).abs(),
            "abs": abs(scale) * (w64.abs() * (size + kl_coef * kl)).sum(), "p": p}


def preference64(logits, targets, offsets, ref, w, beta=0.1, ls=0.0, scale=1.0, lp=None):
    p = None
    if lp is None:
        lp, p = rows64(logits, targets, w)
    on = w != 0
    gain = torch.where(on, w.double() * (lp - (ref.double() if ref is not None else 0.0)), 0.0)
    off = offsets.tolist()
    R = torch.stack([gain[a:b].sum() for a, b in zip(off, off[1:])]) if len(off) > 1 else gain.new_zeros(0)
    z = beta * (R[0::2] - R[1::2])
    softplus = lambda v: torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))  # noqa: E731
    loss = scale * ((1 - ls) * softplus(-z) + ls * softplus(z)).sum()
    dz = scale * (ls * torch.sigmoid(z) - (1 - ls) * torch.sigmoid(-z))
    c = torch.zeros_like(gain)
    for k, (a, b) in enumerate(zip(off, off[1:])):
        c[a:b] = (1 if k % 2 == 0 else -1) * beta * dz[k // 2]
    c = torch.where(on, c * w.double(), 0.0)
    return {"loss": loss, "margins": z, "logprobs": lp, "c": c, "p": p}


def grad64(p, targets, c):
    g = -p * c[:, None]
    if len(c):
        g[torch.arange(len(c), device=c.device), targets.long()] += c
    return g


def assert_logprobs(got, want):
    off = (got.double() - want).abs()
    bound = LP_ABS + LP_REL * want.abs()
    assert bool((off <= bound).all()), f"lp off by {float((off - bound).max())} over the bound"


def assert_grad(got, targets, c, p, size=None, extra=0.0):
    """size: what c's error is relative to (its terms may cancel); extra: added relative error of c."""
    want = grad64(p, targets, c)
    size = (c.abs() if size is None else size)[:, None]
    bound = size * (2e-5 + extra) * p + size * 1e-30 + 2.0 ** -126   # below it fp32 has no full precision
    lp = torch.log(p.gather(1, targets.long()[:, None]))
    at = size * ((2e-5 + extra) * -torch.expm1(lp) + lp.exp() * (LP_ABS + LP_REL * lp.abs()))
    bound = bound.scatter(1, targets.long()[:, None], torch.nan_to_num(at) + 2.0 ** -126)
    if got.dtype == torch.bfloat16:
        bound = bound + want.abs() * 2.0 ** -8 + 1e-38
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} gradient elements off, first at "
                                 f"{bad.nonzero()[:3].tolist()}: {got[bad][:3].tolist()} vs {want[bad][:3].tolist()}")


def assert_close(got, want, tol):
    got, want = float(got), float(want)
    if math.isnan(want) or math.isinf(want):
        assert (math.isnan(got) and math.isnan(want)) or got == want, (got, want)
    else:
        assert abs(got - want) <= tol, (got, want, tol)
