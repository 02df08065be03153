"""token_logprobs, policy_loss and preference_loss against plain 64-bit forms:
types, odd sizes, strides, alignments, masks, special values, streams, graphs."""
import math

import pytest
import torch

import train_util as tu
from allreduce_reduction_emulated_gb300 import losses

pytestmark = pytest.mark.gpu

NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def inputs(dev, T, V, dtype, pad=0, shift=0, seed=0, index=torch.int64, masked=0.25):
    """logits as a view (shift columns into rows of V + pad + shift), targets, old, adv, ref, weights"""
    g = torch.Generator(device=dev).manual_seed(seed)
    whole = torch.randn(T, V + pad + shift, device=dev, generator=g).mul_(3).to(dtype)
    logits = whole[:, shift:shift + V]
    y = torch.randint(0, V, (T,), device=dev, generator=g)
    lp, _ = tu.rows64(logits, y)
    old = (lp + 0.25 * torch.randn(T, device=dev, generator=g)).float()
    # ratios next to a clip bound would let the last bit decide
    r = (lp - old.double()).exp()
    old = torch.where(((r - 1.2).abs() < 1e-3) | ((r - 0.8).abs() < 1e-3), lp.float(), old)
    ref = (lp + 0.3 * torch.randn(T, device=dev, generator=g)).float()
    adv = torch.randn(T, device=dev, generator=g)
    w = torch.rand(T, device=dev, generator=g) + 0.1
    w[torch.rand(T, device=dev, generator=g) < masked] = 0.0
    return logits, y.to(index), old, adv, ref, w


SIZES = [(0, 8), (1, 1), (3, 2), (5, 7), (1, 8), (4, 9), (2, 31), (17, 64), (65, 255), (3, 256), (9, 1000), (700, 33),
         (33, 4097), (2, 16384), (5, 32768), (3, 50001), (2, 131072), (1, 140007), (2, 300001)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,V", SIZES)
def test_logprobs(dev, T, V, dtype):
    logits, y, *_, w = inputs(dev, T, V, dtype, seed=T + V)
    tu.assert_logprobs(losses.token_logprobs(logits, y), tu.rows64(logits, y)[0])
    tu.assert_logprobs(losses.token_logprobs(logits, y, weights=w), tu.rows64(logits, y, w)[0])


def check_policy(logits, y, old, adv, ref, w, kl=0.05, scale=1.0, grad=None, stream=None, source=None):
    source = logits.clone() if source is None else source
    r = losses.policy_loss(logits, y, old, adv, ref_logprobs=ref, weights=w, kl_coef=kl, scale=scale, grad=grad,
                           stream=stream)
    torch.cuda.synchronize()
    want = tu.policy64(source, y, old, adv, ref, w, kl_coef=kl, scale=scale)
    tu.assert_logprobs(r.logprobs, want["logprobs"])
    tol = 2e-5 * float(want["abs"]) + 1e-12
    tu.assert_close(r.loss, want["loss"], tol)
    kl_size, weight = abs(float(want["kl"])), abs(float(want["weight"]))
    tu.assert_close(r.kl, want["kl"], 2e-5 * (kl_size + weight) + 1e-12)
    tu.assert_close(r.clipped, want["clipped"], 1e-6 * weight + 1e-12)
    tu.assert_close(r.weight, want["weight"], 1e-6 * weight + 1e-12)
    assert r.grad.dtype == logits.dtype and r.grad.shape == logits.shape
    if len(y):
        tu.assert_grad(r.grad, y, want["c"], want["p"], want["size"], extra=4e-6)
        assert not bool(r.grad[w == 0].any())
    return r


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,V", SIZES)
def test_policy(dev, T, V, dtype):
    check_policy(*inputs(dev, T, V, dtype, seed=T + 2 * V), scale=0.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("pad,shift,index", [(0, 0, torch.int32), (8, 0, torch.int64), (5, 0, torch.int32),
                                             (0, 1, torch.int64), (3, 3, torch.int64), (8, 8, torch.int32)])
@pytest.mark.parametrize("V", [24, 1001, 20003])
def test_policy_strides_and_alignment(dev, V, pad, shift, index, dtype):
    """Rows at every alignment, in a padded matrix; the gradient (1) into a new
    tensor, (2) into another padded matrix whose padding stays, (3) in place."""
    T = 11
    args = inputs(dev, T, V, dtype, pad, shift, seed=V + pad, index=index)
    first = check_policy(*args).grad
    for off in (0, 1, 2):
        room = torch.full((T, V + 7), 9.0, dtype=dtype, device=dev)
        r = check_policy(*args, grad=room[:, off:off + V])
        assert torch.equal(r.grad, first)
        assert bool((room[:, :off] == 9).all()) and bool((room[:, off + V:] == 9).all())
    source = args[0].clone()
    whole = args[0]._base if args[0]._base is not None else args[0]
    before = whole.clone()
    r = check_policy(*args, grad=args[0], source=source)
    assert r.grad is args[0] and torch.equal(r.grad, first)
    assert torch.equal(whole[:, :shift], before[:, :shift])
    assert torch.equal(whole[:, shift + V:], before[:, shift + V:])


def test_policy_options(dev):
    logits, y, old, adv, ref, w = inputs(dev, 40, 500, torch.float32, seed=4)
    check_policy(logits, y, old, adv, None, w)
    check_policy(logits, y, old, adv, ref, w, kl=0.0)
    check_policy(logits, y, old, adv, ref, w, scale=-2.0 ** -7)
    one = torch.ones_like(w)
    # no weights: the mean over the tokens
    r = losses.policy_loss(logits, y, old, adv)
    want = tu.policy64(logits, y, old, adv, None, one, scale=1 / 40)
    tu.assert_close(r.loss, want["loss"], 2e-5 * float(want["abs"]))
    tu.assert_close(r.weight, 1.0, 1e-6)
    assert float(r.kl) == 0.0
    # one-sided bounds: clip_low 0.1, clip_high 0.5
    r = losses.policy_loss(logits, y, old, adv, ref, w, clip_low=0.1, clip_high=0.5, kl_coef=0.1)
    want = tu.policy64(logits, y, old, adv, ref, w, 0.1, 0.5, 0.1)
    tu.assert_close(r.loss, want["loss"], 2e-5 * float(want["abs"]))
    tu.assert_grad(r.grad, y, want["c"], want["p"], want["size"], extra=4e-6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [130, 9001, 70001])
def test_masked_rows_hold_anything(dev, V, dtype):
    """Rows of weight 0 may hold NaN, infinities, targets outside the row and NaN
    inputs; all rows masked gives zeros."""
    T = 12
    logits, y, old, adv, ref, w = inputs(dev, T, V, dtype, seed=V, masked=0.0)
    w[::3] = 0.0
    clean = check_policy(logits, y, old, adv, ref, w)
    logits, y = logits.clone(), y.clone()
    logits[0] = NAN
    logits[3, ::2] = INF
    logits[6] = -INF
    y[0], y[3], y[6] = -1, V, 1 << 40
    for v in (old, adv, ref):
        v[::3] = NAN
    dirty = losses.policy_loss(logits, y, old, adv, ref, w, kl_coef=0.05)
    for a in ("stats", "grad", "logprobs"):
        assert torch.equal(getattr(clean, a), getattr(dirty, a)), a
    zero = losses.policy_loss(logits, y, old, adv, ref, torch.zeros_like(w), kl_coef=0.05)
    assert not bool(zero.stats.any()) and not bool(zero.grad.any()) and not bool(zero.logprobs.any())
    off = torch.tensor([0, 5, 12], device=dev)
    zero = losses.preference_loss(logits, y, off, ref, torch.zeros_like(w))
    tu.assert_close(zero.loss, math.log(2), 1e-6)
    assert not bool(zero.margins.any()) and not bool(zero.grad.any()) and not bool(zero.logprobs.any())
    assert not bool(losses.token_logprobs(logits, y, torch.zeros_like(w)).any())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [200, 5003, 40000, 100001])
def test_special_logits(dev, V, dtype):
    """Columns masked by -infinity and by the type's lowest value; rows of only
    the lowest value; rows without a distribution (NaN) beside ordinary ones."""
    lowest = torch.finfo(dtype).min
    T = 10
    logits, y, old, adv, ref, w = inputs(dev, T, V, dtype, seed=V, masked=0.0)
    y[:] = torch.arange(T, device=dev)
    logits[:, V // 2:] = -INF
    logits[1, 20:] = lowest
    logits[2, 20:] = -INF
    logits[3] = lowest                    # uniform over V
    logits[4, :] = torch.finfo(dtype).max # uniform too
    old = tu.rows64(logits, y)[0].float()
    ref = old + 0.1
    r = check_policy(logits, y, old, adv, ref, w)
    assert not bool(r.grad[0, V // 2:].any()) and not bool(r.grad[1, 20:].any())
    logits[5, 7] = NAN
    logits[6, 9] = INF
    logits[7] = -INF
    r = losses.policy_loss(logits, y, old, adv, ref, w)
    lp = losses.token_logprobs(logits, y)
    assert torch.equal(torch.isnan(lp), torch.isnan(r.logprobs))
    assert [i for i in range(T) if math.isnan(float(lp[i]))] == [5, 6, 7]
    assert bool(torch.isnan(r.grad[5:8]).all()) and not bool(torch.isnan(r.grad[:5]).any())
    assert not bool(torch.isnan(r.grad[8:]).any()) and math.isnan(float(r.loss))
    # a target of probability zero, without a KL term: ratio 0
    logits, y, old, adv, ref, w = inputs(dev, T, V, dtype, seed=V + 1, masked=0.0)
    logits[:, V - 1] = -INF
    y[:] = V - 1
    adv = adv.abs() + 0.1
    r = losses.policy_loss(logits, y, old.clamp(min=-10), adv, weights=w)
    assert bool((r.logprobs == -INF).all()) and not bool(r.grad.any())
    tu.assert_close(r.loss, 0.0, 0.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_targets_outside_the_row_give_nan(dev, dtype):
    for V in (50, 33000):
        logits, y, old, adv, ref, w = inputs(dev, 6, V, dtype, masked=0.0)
        y[1], y[2], y[3] = V, -100, 1 << 33
        r = losses.policy_loss(logits, y, old, adv, weights=w)
        bad = torch.tensor([False, True, True, True, False, False], device=dev)
        assert torch.equal(torch.isnan(losses.token_logprobs(logits, y)), bad)
        assert torch.equal(torch.isnan(r.logprobs), bad)
        assert torch.equal(torch.isnan(r.grad).all(1), bad) and torch.equal(torch.isnan(r.grad).any(1), bad)


def lengths_to_offsets(n, dev, dtype=torch.int64):
    return torch.tensor([0] + [sum(n[:i + 1]) for i in range(len(n))], device=dev, dtype=dtype)


def check_preference(logits, y, off, ref, w, beta=0.1, ls=0.0, scale=None, grad=None):
    source = logits.clone()
    pairs = len(off) // 2
    r = losses.preference_loss(logits, y, off, ref, w, beta=beta, label_smoothing=ls, scale=scale, grad=grad)
    s = 1 / max(1, pairs) if scale is None else scale
    want = tu.preference64(source, y, off, ref, w, beta, ls, s)
    tu.assert_logprobs(r.logprobs, want["logprobs"])
    # a margin adds beta w times each row's error
    lp = want["logprobs"].abs().max() if len(y) else 0.0
    size = float(beta * w.sum()) * (tu.LP_ABS + 2 * tu.LP_REL * float(lp)) + 1e-7
    off_z = (r.margins.double() - want["margins"]).abs()
    assert bool((off_z <= size + 1e-6 * want["margins"].abs()).all())
    tu.assert_close(r.loss, want["loss"], abs(s) * pairs * size + 1e-6 * abs(float(want["loss"])) + 1e-12)
    if len(y):
        # sigmoid(-z) is relative to z's error
        tu.assert_grad(r.grad, y, want["c"], want["p"], extra=2 * size)
    return r


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 7, 64, 1003, 32768, 50001])
@pytest.mark.parametrize("lengths", [(1, 1), (3, 5), (0, 4), (4, 0), (0, 0), (7, 2, 1, 30), (5, 5, 0, 0, 2, 9)])
def test_preference(dev, lengths, V, dtype):
    T = sum(lengths)
    logits, y, _, _, ref, w = inputs(dev, T, V, dtype, seed=V + T, index=torch.int32)
    off = lengths_to_offsets(lengths, dev, torch.int32 if V % 2 else torch.int64)
    check_preference(logits, y, off, ref, w)
    check_preference(logits, y, off, None, w, beta=0.02, ls=0.1, scale=0.25)
    check_preference(logits, y, off, ref, w, grad=logits)


def test_preference_long_sequences(dev):
    lengths = (900, 1300, 1, 2049)
    logits, y, _, _, ref, w = inputs(dev, sum(lengths), 300, torch.float32, pad=5)
    check_preference(logits, y, lengths_to_offsets(lengths, dev), ref, w, beta=0.01)


def test_preference_many_pairs(dev):
    lengths = tuple(i % 4 for i in range(2 * 1500))
    logits, y, _, _, ref, w = inputs(dev, sum(lengths), 40, torch.bfloat16)
    check_preference(logits, y, lengths_to_offsets(lengths, dev), ref, w)


def test_preference_rows_of_no_sequence_and_no_pairs(dev):
    logits, y, _, _, ref, w = inputs(dev, 20, 90, torch.float32, masked=0.0)
    off = torch.tensor([3, 8, 15], device=dev)
    r = check_preference(logits, y, off, ref, w)
    assert not bool(r.grad[:3].any()) and not bool(r.grad[15:].any()) and bool(r.grad[3:15].any())
    r = losses.preference_loss(logits, y, off[:1], ref, w)
    assert float(r.loss) == 0.0 and r.margins.numel() == 0 and not bool(r.grad.any())
    # offsets outside [0, tokens] are clamped
    far = losses.preference_loss(logits, y, torch.tensor([-5, 8, 1 << 40], device=dev), ref, w)
    near = losses.preference_loss(logits, y, torch.tensor([0, 8, 20], device=dev), ref, w)
    assert torch.equal(far.margins, near.margins) and torch.equal(far.grad, near.grad)


@pytest.mark.parametrize("z", [300.0, -300.0, 1e5, -1e5])
def test_preference_extreme_margins(dev, z):
    """The loss and its derivative stay finite and right far from zero."""
    logits, y, _, _, ref, w = inputs(dev, 2, 50, torch.float32, masked=0.0)
    w[:] = 1.0
    lp, _ = tu.rows64(logits, y)
    ref = lp.float()
    ref[0] -= z / 0.1
    check_preference(logits, y, torch.tensor([0, 1, 2], device=dev), ref, w)


def test_preference_targets_of_probability_zero(dev):
    """A rejected answer with a token of probability zero: margin infinite, loss and
    gradient 0; a chosen one: loss infinite, gradient that of the linear branch."""
    logits, y, _, _, ref, w = inputs(dev, 4, 70, torch.float32, masked=0.0)
    w[:] = 1.0
    off = torch.tensor([0, 2, 4], device=dev)
    for row, loss, dz in ((3, 0.0, 0.0), (0, INF, -1.0)):
        x, t = logits.clone(), y.clone()
        t[row] = 69
        x[:, 69] = -1.0
        x[row, 69] = -INF
        r = losses.preference_loss(x, t, off, ref, w, beta=0.1)
        tu.assert_close(r.loss, loss, 0.0)
        assert float(r.margins) == (INF if dz == 0 else -INF) and float(r.logprobs[row]) == -INF
        lp, p = tu.rows64(x, t, w)
        c = 0.1 * dz * torch.tensor([1.0, 1.0, -1.0, -1.0], device=dev, dtype=torch.float64)
        want = tu.grad64(p, t, c)
        assert bool(((r.grad.double() - want).abs() <= 1e-5 * want.abs() + 1e-12).all())


@pytest.mark.parametrize("length", [1, 255, 600, 1025])
def test_preference_of_equal_answers(dev, length):
    """The same answer on both sides (rows alike in their lines), without a reference: every difference is exactly
    0, and so is the margin, however long the answers are; the loss is log 2."""
    logits, y, _, _, _, _ = inputs(dev, length, 1024, torch.float32, masked=0.0)
    logits, y = logits.repeat(2, 1), y.repeat(2)
    r = losses.preference_loss(logits, y, torch.tensor([0, length, 2 * length], device=dev), beta=0.5)
    assert float(r.margins) == 0.0
    tu.assert_close(r.loss, math.log(2.0), 2 ** -22)
    assert torch.equal(r.grad[:length], -r.grad[length:])


@pytest.mark.parametrize("rows,vocab", [(1500, 9001), (3000, 30000), (5200, 50001)])
def test_preference_around_l2(dev, rows, vocab):
    """Matrices of 27, 180 and 520 MB, around what L2 can keep for the gradient."""
    logits, y, _, _, ref, w = inputs(dev, rows, vocab, torch.bfloat16)
    n = rows // 6
    check_preference(logits, y, torch.arange(0, rows + 1, n, device=dev)[:7], ref, w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 1001, 9001, 40003])
def test_gradients_at_other_alignments(dev, V, dtype):
    """Gradients at every distance from the logits' alignment, targets at every place of
    a slot and of a warp's stores: what is beside the rows stays."""
    T = 24
    logits, y, old, adv, ref, w = inputs(dev, T, V, dtype, seed=V)
    w[:] = 1.0
    y[:] = torch.arange(T, device=dev) * 33 % V
    N = 16 // logits.element_size()
    off = torch.tensor([0, 5, 11, 20, T], device=dev)
    for shift in range(1, N):
        room = torch.full((T, V + N), 9.0, dtype=dtype, device=dev)
        check_preference(logits, y, off, ref, w, grad=room[:, shift:shift + V])
        assert bool((room[:, :shift] == 9).all()) and bool((room[:, shift + V:] == 9).all())
        room[:] = 9.0
        check_policy(logits, y, old, adv, ref, w, grad=room[:, shift:shift + V])
        assert bool((room[:, :shift] == 9).all()) and bool((room[:, shift + V:] == 9).all())


# slots of 16 bytes at which the policy loss changes its shape (blocks, clusters, registers per thread)
SHAPES = [512, 1024, 1536, 2048, 2560, 3584, 4096, 5120, 8192, 10240, 12288, 16384, 20480, 32768, 49152, 65536]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("slots", SHAPES)
def test_policy_shapes(dev, slots, dtype):
    """Rows that just fill a shape, begin at an odd element, or need one slot more."""
    N = 16 // (4 if dtype == torch.float32 else 2)
    for V, pad, shift in ((slots * N, 0, 0), (slots * N - 2 * N, 1, 3), (slots * N + 1, 0, 0)):
        check_policy(*inputs(dev, 5, V, dtype, pad, shift, seed=slots))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(5000, 700), (3100, 4099), (2500, 9001), (1300, 20011), (700, 50003)])
def test_many_rows(dev, T, V, dtype):
    """Enough rows that a cluster takes several, masked ones among them; in place too."""
    logits, y, old, adv, ref, w = inputs(dev, T, V, dtype, seed=T)
    first = check_policy(logits, y, old, adv, ref, w)
    tu.assert_logprobs(losses.token_logprobs(logits, y, w), tu.rows64(logits, y, w)[0])
    off = lengths_to_offsets((T // 4, T // 2, 3, T // 8), dev)
    check_preference(logits, y, off, ref, w, beta=0.001)
    again = losses.policy_loss(logits, y, old, adv, ref, w, kl_coef=0.05, scale=1.0, grad=logits)
    assert torch.equal(again.grad, first.grad) and torch.equal(again.stats, first.stats)


@pytest.mark.parametrize("op", ["policy", "preference"])
def test_gradient_against_differences(dev, op):
    """The kernel's gradient against central differences of the 64-bit loss along
    random directions (step 1e-5: truncation and rounding under 1e-8 relative)."""
    T, V = 14, 301
    logits, y, old, adv, ref, w = inputs(dev, T, V, torch.float32, seed=5)
    off = torch.tensor([0, 4, 9, 11, 14], device=dev)
    if op == "policy":
        grad = losses.policy_loss(logits, y, old, adv, ref, w, kl_coef=0.1).grad
        loss = lambda x: tu.policy64(x, y, old, adv, ref, w, kl_coef=0.1)["loss"]  # noqa: E731
    else:
        grad = losses.preference_loss(logits, y, off, ref, w, label_smoothing=0.1, scale=1.0).grad
        loss = lambda x: tu.preference64(x, y, off, ref, w, ls=0.1)["loss"]  # noqa: E731
    g = torch.Generator(device=dev).manual_seed(1)
    x = logits.double()
    for _ in range(8):
        v = torch.randn(T, V, device=dev, generator=g, dtype=torch.float64)
        h = 1e-5
        diff = float((loss(x + h * v) - loss(x - h * v)) / (2 * h))
        size = float((grad.double() * v).abs().sum())
        assert abs(float((grad.double() * v).sum()) - diff) <= 3e-5 * size


def test_offsets_past_32_bits(dev):
    """A matrix of more than 2^32 elements: only rows at its two ends count."""
    T, V = 66000, 66001
    logits = torch.zeros(T, V, dtype=torch.bfloat16, device=dev)
    keep = [0, 1, T // 2, T - 2, T - 1]
    g = torch.Generator(device=dev).manual_seed(3)
    logits[keep] = torch.randn(len(keep), V, device=dev, generator=g).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), device=dev, generator=g)
    w = torch.zeros(T, device=dev)
    w[keep] = 1.0
    small, ys, ws = logits[keep].clone(), y[keep].clone(), w[keep].clone()
    lp, _ = tu.rows64(small, ys)
    old = torch.zeros(T, device=dev)
    old[keep] = lp.float() - 0.1
    adv = torch.ones(T, device=dev)
    tu.assert_logprobs(losses.token_logprobs(logits, y, w)[keep], lp)
    r = losses.policy_loss(logits, y, old, adv, weights=w, grad=logits)
    want = tu.policy64(small, ys, old[keep], adv[keep], None, ws)
    tu.assert_close(r.loss, want["loss"], 2e-5 * float(want["abs"]))
    tu.assert_grad(logits[keep], ys, want["c"], want["p"], want["size"], extra=4e-6)
    logits[keep] = 0
    assert int(torch.count_nonzero(logits)) == 0


def test_other_streams_repeats_and_graphs(dev):
    """The same bits on the default stream, on a side stream (given and current),
    behind other work, and replayed from a graph on new data."""
    logits, y, old, adv, ref, w = inputs(dev, 300, 8193, torch.bfloat16, seed=8)
    off = torch.tensor([0, 70, 150, 220, 300], device=dev)
    f = lambda **kw: losses.policy_loss(logits, y, old, adv, ref, w, kl_coef=0.1, **kw)  # noqa: E731
    h = lambda **kw: losses.preference_loss(logits, y, off, ref, w, **kw)  # noqa: E731
    a, b = f(), h()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for run in range(3):
        if run == 0:
            c, d = f(stream=side), h(stream=side)
        elif run == 1:
            c, d = f(stream=side.cuda_stream), h(stream=side.cuda_stream)
        else:
            with torch.cuda.stream(side):
                c, d = f(), h()
        side.synchronize()
        assert torch.equal(a.stats, c.stats) and torch.equal(a.grad, c.grad) and torch.equal(a.logprobs, c.logprobs)
        assert torch.equal(b.loss, d.loss) and torch.equal(b.grad, d.grad) and torch.equal(b.margins, d.margins)
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c, d, e = f(), h(), losses.token_logprobs(logits, y)
    for seed in (8, 9):
        new = inputs(dev, 300, 8193, torch.bfloat16, seed=seed)[0]
        logits.copy_(new)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        a, b = f(), h()
        assert torch.equal(a.stats, c.stats) and torch.equal(a.grad, c.grad) and torch.equal(a.logprobs, c.logprobs)
        assert torch.equal(b.loss, d.loss) and torch.equal(b.grad, d.grad) and torch.equal(b.margins, d.margins)
        assert torch.equal(e, losses.token_logprobs(logits, y))


def test_back_to_back_calls_keep_stream_order(dev):
    """Each call reads what the one before it wrote (in-place gradients), with no host wait."""
    logits, y, old, adv, ref, w = inputs(dev, 64, 2050, torch.float32, seed=2, masked=0.0)
    x = logits.clone()
    for _ in range(5):
        losses.policy_loss(x, y, old, adv, weights=w, grad=x)
        losses.preference_loss(x, y, torch.tensor([0, 30, 64], device=dev), ref, w, grad=x, beta=1.0)
    z = logits.clone()
    for _ in range(5):
        z = losses.policy_loss(z, y, old, adv, weights=w).grad.clone()
        torch.cuda.synchronize()
        z = losses.preference_loss(z, y, torch.tensor([0, 30, 64], device=dev), ref, w, beta=1.0).grad.clone()
        torch.cuda.synchronize()
    assert torch.equal(x, z)
