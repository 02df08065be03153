"""Plain 64-bit form of the orthogonalised update, and its tolerance.

Between the products X, A and B = b A + c A^2 are fp16 times a power of two: each element is off by at most
half a step, 2^-11 of its value (what underflows is 2^-25 of a matrix' bound of 2^13 or less and does not
count).  The roundings are independent, so that a matrix is off by at most e = 2^-11 / sqrt(3) = 2.8e-4 of its
2-norm (Frobenius).  One step X <- f(X) carries an error of X on by at most the largest slope of
p(s) = a s + b s^3 + c s^5 that matters, relative to how the step grows X itself: while the singular values are small both
are a, and the relative error stays; where they have reached 0.7 .. 1.2 the slope lies between -1.6 and 2 of values
that stay the same.  A's and B's own roundings enter as B's error times X: |b| s^2 + 2 |c| s^4 <= 11 e / sqrt(3)
where s = 1, in random directions.  Over five steps, of which the last three are in that range, the errors add in squares to
less than e sqrt(2^2 + 2^4 + 2^6 + (11 / sqrt(3))^2 (1 + 2^2 + 2^4) / 8) = 14 e = 4e-3 at the very most, where all singular
values sit at the worst place; over the range of values of a matrix the mean square slope is below 1 and
1e-3 is what adds up.  The tests hold the result to 5e-3 with the half step of bf16 (2^-8 / sqrt(3) =
2.3e-3) in it.
"""
import torch

TOL = 5e-3


def update64(g, m=None, beta=0.95, nesterov=True, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, scale=1.0):
    """(update, momentum) of a matrix or a stack of them."""
    u = g.double()
    if m is not None:
        m = beta * m.double() + u
        u = u + beta * m if nesterov else m
    a, b, c = coefficients
    tall = u.shape[-2] > u.shape[-1]
    x = u.transpose(-1, -2) if tall else u
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        A = x @ x.transpose(-1, -2)
        x = a * x + (b * A + c * A @ A) @ x
    return scale * (x.transpose(-1, -2) if tall else x), m


def assert_update(got, want, tol=TOL):
    assert got.shape == want.shape
    off = (got.double() - want).flatten(-2).norm(dim=-1)
    size = want.flatten(-2).norm(dim=-1)
    assert bool((off <= tol * size + 1e-30).all()), f"off by {float((off / size).max())} of the 2-norm"
