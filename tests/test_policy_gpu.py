"""policy_loss where its terms are far apart in size: terms of weight 0, near-certain tokens,
very long rows, many rows."""
import math

import pytest
import torch

import train_util as tu
from allreduce_reduction_emulated_gb300 import losses

pytestmark = pytest.mark.gpu
INF = math.inf
BOTH = [torch.float32, torch.bfloat16]
IDS = ["f32", "bf16"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.mark.parametrize("V", [300, 40000, 600001])
def test_kl_term_of_coefficient_zero_is_left_out(dev, V):
    """A reference given for the statistic alone: where e^d is infinite the statistic is, not the loss."""
    g = torch.Generator(device=dev).manual_seed(V)
    T = 6
    logits = torch.randn(T, V, device=dev, generator=g)
    y = torch.arange(T, device=dev)
    logits[2, 2] = -200.0
    old = losses.token_logprobs(logits, y) - 0.1
    adv = torch.randn(T, device=dev, generator=g)
    ref = old.clone()
    ref[2] = 0.0
    plain = losses.policy_loss(logits, y, old, adv)
    r = losses.policy_loss(logits, y, old, adv, ref_logprobs=ref, kl_coef=0.0)
    assert torch.equal(r.loss, plain.loss) and torch.equal(r.grad, plain.grad)
    assert float(r.kl) == INF and math.isfinite(float(r.loss))


@pytest.mark.parametrize("dtype", BOTH, ids=IDS)
@pytest.mark.parametrize("T,V", [(3000, 3000), (2000, 9000), (1200, 50003), (300, 131072)])
def test_in_place_behind_masked_rows(dev, T, V, dtype):
    """In place where the first rows that a cluster works on are masked: the same bits as in a new gradient."""
    g = torch.Generator(device=dev).manual_seed(V)
    logits = (3 * torch.randn(T, V, device=dev, generator=g)).to(dtype)
    y = torch.randint(0, V, (T,), device=dev, generator=g)
    adv = torch.randn(T, device=dev, generator=g)
    old = losses.token_logprobs(logits, y) + 0.1
    for masked in (1, 2, 3, 5):
        w = (torch.arange(T, device=dev) % (masked + 1) == masked).float()
        first = losses.policy_loss(logits, y, old, adv, weights=w)
        x = logits.clone()
        again = losses.policy_loss(x, y, old, adv, weights=w, grad=x)
        assert torch.equal(again.grad, first.grad) and torch.equal(again.stats, first.stats)
        assert torch.equal(again.logprobs, first.logprobs)


@pytest.mark.parametrize("dtype", BOTH, ids=IDS)
@pytest.mark.parametrize("low", [-14.0, -18.0, -24.0])
@pytest.mark.parametrize("V", [5003, 9000, 20011, 50003, 131072, 262100])
def test_near_certain_tokens(dev, V, low, dtype):
    """One logit far above all others: lp = -log(1 + rest), the rest between 1e-7 and 0.3.  A thread
    adds at most 32 of a row's terms (64 from 65536 columns on) to the maximum's 1 and may lose them (32 / V of
    the rest); 1% of it covers that and what e^z rounds.  token_logprobs agrees, so that ratios of freshly scored tokens are 1, and the
    target's gradient balances the other columns'."""
    T = 13
    g = torch.Generator(device=dev).manual_seed(V)
    logits = (low + torch.rand(T, V, device=dev, generator=g)).to(dtype)
    y = torch.arange(T, device=dev) * 389 % V
    logits[torch.arange(T, device=dev), y] = 0.0
    x = logits.double()
    x[torch.arange(T, device=dev), y] = -INF
    rest = x.exp().sum(1)
    want = -torch.log1p(rest)
    fresh = losses.token_logprobs(logits, y)
    adv = torch.ones(T, device=dev)
    r = losses.policy_loss(logits, y, fresh, adv, scale=-1.0)
    assert bool(((r.logprobs.double() - want).abs() <= 0.01 * want.abs()).all())
    assert bool(((fresh.double() - want).abs() <= 0.01 * want.abs()).all())
    assert bool(((r.logprobs - fresh).double().abs() <= 0.01 * want.abs()).all())
    # grad = r ([j = y] - p_j): 1 - p of the target, and the others' sum
    p = rest / (1 + rest)
    at = r.grad[torch.arange(T, device=dev), y].double()
    assert bool(((at - p).abs() <= (0.01 + 2.0 ** -8) * p).all())
    others = r.grad.double().sum(1) - at
    assert bool(((others + p).abs() <= (0.01 + 2.0 ** -8) * p).all())


@pytest.mark.parametrize("dtype", BOTH, ids=IDS)
@pytest.mark.parametrize("V", [600001, (1 << 21) + 3, 1 << 24])
def test_very_long_rows(dev, V, dtype):
    """Rows that no cluster holds: flat ones, ones with a hundred equal maxima, near-certain tokens.  The bounds are
    those of short rows: sums are carried over."""
    T = 5
    x = torch.full((T, V), -20.0, dtype=dtype, device=dev)
    x[0] = 1.5
    x[1, ::2] = -19.0
    x[2, ::V // 100] = 0.0
    x[3, 17], x[4, V - 1] = 8.0, 4.0
    y = torch.tensor([3, 8, V // 100, 17, V - 1], device=dev)
    w = torch.ones(T, device=dev)
    want, p = tu.rows64(x, y)
    fresh = losses.token_logprobs(x, y)
    tu.assert_logprobs(fresh, want)
    r = losses.policy_loss(x, y, fresh, w, scale=1.0)
    tu.assert_logprobs(r.logprobs, want)
    assert bool(((r.logprobs.double() - want)[3:].abs() <= 0.01 * want[3:].abs()).all())
    assert bool(((r.logprobs - fresh).double()[3:].abs() <= 0.01 * want[3:].abs()).all())
    tu.assert_grad(r.grad, y, tu.policy64(x, y, fresh, w, None, w)["c"], p, w.double(), extra=4e-6)


def test_sums_of_many_rows(dev):
    """Sums where every rounding goes the same way.  At most 32 rows are added up one after the other (16.5 2^-24 of
    their sum), the clusters' sums are carried over in each thread and added in a tree (5 + 8 additions), the scale
    rounds once: under 32 2^-24 = 2e-6."""
    T = 3_000_001
    x = torch.zeros(T, 8, device=dev)
    y = torch.zeros(T, dtype=torch.int32, device=dev)
    lp = losses.token_logprobs(x[:1], y[:1])[0]
    old = lp.expand(T).contiguous()
    adv = torch.ones(T, device=dev)
    for w in (0.3, 0.7, 0.1, 0.45):
        weights = torch.full((T,), w, device=dev)
        r = losses.policy_loss(x, y, old, adv, weights=weights)
        want = float(weights[0]) * T
        assert abs(float(r.weight) - want) <= 2e-6 * want, (w, float(r.weight) / want - 1)
        assert abs(float(r.loss) + want) <= 2.1e-6 * want, (w, float(r.loss) / want + 1)


def test_preference_sums_of_many_pairs_and_tokens(dev):
    """The loss over many pairs and a margin over a long sequence, every addition rounding the same way: carried over
    in each thread, then a tree (13 additions): under 16 2^-24 = 1e-6."""
    pairs = 400_000
    x = torch.zeros(2 * pairs, 2, device=dev)
    y = torch.zeros(2 * pairs, dtype=torch.int32, device=dev)
    off = torch.arange(2 * pairs + 1, device=dev)
    r = losses.preference_loss(x, y, off, scale=1.0)
    want = pairs * math.log(2.0)
    assert abs(float(r.loss) - want) <= 1.2e-6 * want, float(r.loss) / want - 1
    for ref in (-0.3, -0.45, -1.1):
        refs = torch.full((2 * pairs,), ref, device=dev)
        off = torch.tensor([0, 2 * pairs, 2 * pairs], device=dev)
        r = losses.preference_loss(x, y, off, refs, beta=1.0)
        gain = float((r.logprobs[0] - refs[0]).double()) * 2 * pairs
        assert abs(float(r.margins) - gain) <= 1e-6 * abs(gain), (ref, float(r.margins) / gain - 1)
