"""Plain 64-bit forms of the expert products, and tolerances, for their tests.

A product of two bf16 values is exact in fp32.  The tensor cores add a slice of 16 of them
to the accumulator at a time: ceil(k / 16) additions, each off by at most a whole unit
(2^-23, whether it rounds or cuts) of a partial sum that is at most S = sum |a| |b|; the 16 of a
slice are aligned to the largest and add no more than one unit each.  So a sum is within
(ceil(k / 16) + 16) 2^-23 S, and a bf16 result within half a step (2^-8) of its value more.
"""
import torch


def ranges(offsets, rows):
    """[(first row, end)] of each expert: clamped, never falling."""
    off, at, out = [min(max(int(v), 0), rows) for v in offsets.tolist()], 0, []
    for a, b in zip(off, off[1:]):
        at = max(at, a)
        out.append((at, max(at, b)))
    return out


def product64(x, w, offsets):
    """(y, S): zeros for rows of no expert."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=x.device)
    S = torch.zeros_like(y)
    for e, (a, b) in enumerate(ranges(offsets, len(x))):
        if a < b:
            y[a:b] = x[a:b].double() @ w[e].double().t()
            S[a:b] = x[a:b].double().abs() @ w[e].double().abs().t()
    return y, S


def weight_gradient64(dy, x, offsets, experts):
    dw = torch.zeros(experts, dy.shape[1], x.shape[1], dtype=torch.float64, device=x.device)
    S = torch.zeros_like(dw)
    for e, (a, b) in enumerate(ranges(offsets, len(x))):
        if a < b:
            dw[e] = dy[a:b].double().t() @ x[a:b].double()
            S[e] = dy[a:b].double().abs().t() @ x[a:b].double().abs()
    return dw, S


def assert_sum(got, want, S, k):
    tol = (-(-k // 16) + 16) * 2.0 ** -23 * S
    if got.dtype == torch.bfloat16:
        tol = tol + (want.abs() + tol) * 2.0 ** -8 + 1e-38
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[:3].tolist()}: "
                                 f"{got[bad][:3].tolist()} vs {want[bad][:3].tolist()}, tolerance {tol[bad][:3].tolist()}")
