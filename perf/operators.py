"""The operators at the two ends of the data-parallel step, and what is measured of them.

Before the all-reduce: the log-probabilities of tokens under a policy, the
clipped policy loss with a KL term and the preference loss over paired
sequences, each with the gradient of the logits.  After it: the global norm
of the reduced gradients, and clipping.

    op = "logprobs"    logp[t] = x[t, y_t] - logsumexp(x[t, :])
    op = "policy"      loss, KL and clipped share, gradient of the logits, logp
    op = "preference"  loss, margins, gradient of the logits, logp
    op = "clip"        norm over all tensors and the clipped gradients

own = False runs plain torch operations in 32 bits; own = True the package's
operators.
"""
import math
import random

import torch

own = False

MAX_NORM = 1.0        # clip: the usual bound of a training loop
EPS = 1e-6            # clip: max_norm / (norm + EPS)
CLIP = 0.2            # policy: ratios are clipped to [1 - CLIP, 1 + CLIP]
KL = 0.05             # policy: weight of the KL term where the case has one
BETA = 0.1            # preference: weight of the paired log ratios
ES = {"float32": 4, "bfloat16": 2}
# the four weight matrices of one of the 24 layers of the 1.2B-parameter gradient workload
LAYER = (2048 * 8192, 8192 * 2048, 2048 * 6144, 2048 * 2048)


def listed():
    return [
        # one sampled token scored as it is generated
        {"name": "logprobs 1x32768 bf16", "op": "logprobs", "tokens": 1, "vocab": 32768, "dtype": "bfloat16", "pad": 0},
        # a batch of rollouts scored by the reference policy
        {"name": "logprobs 4096x131072 bf16", "op": "logprobs", "tokens": 4096, "vocab": 131072, "dtype": "bfloat16",
         "pad": 0},
        # an odd vocabulary in rows padded to 64 columns, 32-bit logits
        {"name": "logprobs 1000x50001 f32", "op": "logprobs", "tokens": 1000, "vocab": 50001, "dtype": "float32",
         "pad": 47},
        # the last micro-batch of a short answer: latency
        {"name": "policy 16x32768 bf16", "op": "policy", "tokens": 16, "vocab": 32768, "dtype": "bfloat16", "pad": 0,
         "masked": 0.0, "kl": True, "dead": 0},
        # an ordinary micro-batch, the prompts' tokens masked
        {"name": "policy 4096x32768 bf16", "op": "policy", "tokens": 4096, "vocab": 32768, "dtype": "bfloat16",
         "pad": 0, "masked": 0.3, "kl": True, "dead": 0},
        # a large micro-batch over a large vocabulary whose last columns are unused
        {"name": "policy 8192x131072 bf16", "op": "policy", "tokens": 8192, "vocab": 131072, "dtype": "bfloat16",
         "pad": 0, "masked": 0.0, "kl": True, "dead": 256},
        # odd vocabulary without padding: every row starts at another alignment; 32-bit logits, no reference policy
        {"name": "policy 1111x50001 f32", "op": "policy", "tokens": 1111, "vocab": 50001, "dtype": "float32", "pad": 0,
         "masked": 0.1, "kl": False, "dead": 0},
        # two short pairs
        {"name": "preference 2x24 32768 bf16", "op": "preference", "pairs": 2, "shortest": 8, "longest": 24,
         "vocab": 32768, "dtype": "bfloat16", "pad": 0, "masked": 0.0},
        # a batch of pairs with answers of very different lengths, prompts masked, an odd vocabulary
        {"name": "preference 8x300 50001 bf16", "op": "preference", "pairs": 8, "shortest": 30, "longest": 300,
         "vocab": 50001, "dtype": "bfloat16", "pad": 0, "masked": 0.25},
        # long answers over a large vocabulary
        {"name": "preference 4x1024 131072 bf16", "op": "preference", "pairs": 4, "shortest": 700, "longest": 1024,
         "vocab": 131072, "dtype": "bfloat16", "pad": 0, "masked": 0.0},
        # the gradients of a small model: many small odd tensors, below the bound (nothing to scale)
        {"name": "clip 37 tensors 200k f32", "op": "clip", "tensors": 37, "total": 200_003, "dtype": "float32",
         "layers": 0},
        # all gradients of the 1.2B-parameter workload, its 24 layers of four matrices
        {"name": "clip 96 tensors 1.2G f32", "op": "clip", "tensors": 96, "total": 24 * sum(LAYER), "dtype": "float32",
         "layers": 24},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "policy", "preference", "clip"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    if op == "clip":
        total = _log_between(rng, 20_000, 600_000_000)
        return {"op": op, "tensors": rng.randint(1, min(400, 1 + total // 64)), "total": total, "dtype": dtype,
                "layers": 0}
    most = 8192 * 131072 * 2 // ES[dtype]           # elements of the largest listed case
    vocab = _log_between(rng, 4000, 140_000)
    if rng.random() < 0.6:
        vocab = -(-vocab // 64) * 64                # most vocabularies are padded to whole vectors
    case = {"op": op, "vocab": vocab, "dtype": dtype, "pad": rng.choice([0, 0, 0, 8, 13])}
    if op == "preference":
        most = most // 2                            # its rows are read twice
        pairs = _log_between(rng, 1, 32)
        longest = max(4, min(_log_between(rng, 8, 2048), most // (2 * pairs * vocab)))
        case |= {"pairs": pairs, "shortest": rng.randint(1, longest), "longest": longest}
    else:
        case |= {"tokens": max(1, min(_log_between(rng, 1, 16384), most // vocab))}
    if op != "logprobs":
        case |= {"masked": rng.choice([0.0, round(rng.uniform(0.0, 0.6), 3)])}
    if op == "policy":
        case |= {"kl": rng.random() < 0.6, "dead": rng.choice([0, 0, min(vocab // 2, 101)])}
    return case


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """Rows of each of the 2 * pairs sequences: chosen, rejected, chosen, ...; the same for every seed."""
    r = random.Random(case["pairs"] * 1_000_003 + case["longest"])
    n = [r.randint(case["shortest"], case["longest"]) for _ in range(2 * case["pairs"])]
    n[r.randrange(len(n))] = case["longest"]
    return n


def _tokens(case):
    return sum(_lengths(case)) if case["op"] == "preference" else case["tokens"]


def _masked(case):
    return int(_tokens(case) * case.get("masked", 0.0))


def _sizes(case):
    """Elements of each gradient tensor."""
    if case["layers"]:
        return [n for _ in range(case["layers"]) for n in LAYER]
    r = random.Random(case["total"])
    cuts = sorted(r.sample(range(1, case["total"]), case["tensors"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["total"]])]


def _chunk_logp(logits, targets, dtype):
    """logp of every row, a few rows at a time (for the inputs that a rollout has recorded)."""
    rows = max(1, (1 << 27) // logits.shape[1])
    parts = []
    for a in range(0, logits.shape[0], rows):
        x = logits[a:a + rows].to(dtype)
        parts.append(x.gather(1, targets[a:a + rows, None]).squeeze(1) - torch.logsumexp(x, 1))
    return torch.cat(parts)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = getattr(torch, case["dtype"])
    if case["op"] == "clip":
        grads = torch.empty(case["total"], dtype=dtype, device="cuda").normal_(0.0, 1e-3, generator=gen)
        state = {"case": case, "grads": grads, "out": torch.empty_like(grads)}
        if own:
            from allreduce_reduction_emulated_gb300.clipping import GradClipper
            sizes = _sizes(case)
            state["clipper"] = GradClipper(grads.split(sizes), out=state["out"].split(sizes))
        return state
    T, V = _tokens(case), case["vocab"]
    logits = torch.empty(T, V + case["pad"], dtype=dtype, device="cuda").normal_(0.0, 2.0, generator=gen)[:, :V]
    live = V - case.get("dead", 0)
    if live < V:
        logits[:, live:] = -math.inf
    targets = torch.randint(0, live, (T,), device="cuda", generator=gen)
    # the sampled tokens are likely ones
    likely = torch.empty(T, device="cuda").normal_(math.log(V) + 1.5, 1.5, generator=gen)
    logits[torch.arange(T, device="cuda"), targets] = likely.to(dtype)
    state = {"case": case, "logits": logits, "targets": targets}
    if case["op"] == "logprobs":
        return state
    logp = _chunk_logp(logits, targets, torch.float32)
    keep = torch.ones(T, device="cuda")
    keep[torch.randperm(T, device="cuda", generator=gen)[:_masked(case)]] = 0.0
    noise = torch.empty(2, T, device="cuda").normal_(generator=gen)
    if case["op"] == "policy":
        # log ratios of a few updates; none within 0.002 of the clip bounds, where the derivative
        # jumps and the last bit of logp would decide which side a token is on
        u = 0.15 * noise[0]
        r = u.exp()
        u[((r - (1 + CLIP)).abs() < 0.002) | ((r - (1 - CLIP)).abs() < 0.002)] = 0.0
        state["old"] = logp - u
        state["ref"] = logp + 0.2 * noise[1] if case["kl"] else None
        state["advantages"] = torch.empty(T, device="cuda").normal_(0.3, 1.0, generator=gen)
        state["weights"] = keep / max(1, T - _masked(case))
        return state
    n = torch.tensor(_lengths(case), device="cuda")
    side = torch.tensor([1.0, -1.0], device="cuda").repeat(case["pairs"]).repeat_interleave(n)
    each = n.repeat_interleave(n).float()
    # the policy has moved a few nats towards the chosen answers
    state["ref"] = logp - 4.0 * side / each + noise[0] / each.sqrt()
    state["weights"] = keep
    state["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)])
    return state


# ------------------------------------------------------------------ the plain forms

def _rows(logits, targets):
    """logp and the probabilities of every row."""
    x = logits.float()
    m = x.amax(1, keepdim=True)
    e = (x - m).exp()
    s = e.sum(1, keepdim=True)
    logp = (x.gather(1, targets[:, None]) - m - s.log()).squeeze(1)
    return logp, e / s


def _grad(p, targets, c, dtype):
    """c[t] * (onehot(y_t) - p[t, :]), rounded once."""
    return (-p * c[:, None]).scatter_add_(1, targets[:, None], c[:, None]).to(dtype)


def _plain_logprobs(s):
    return _rows(s["logits"], s["targets"])[0]


def _plain_policy(s):
    w, A = s["weights"], s["advantages"]
    logp, p = _rows(s["logits"], s["targets"])
    logp = torch.where(w != 0, logp, 0.0)
    r = (logp - s["old"]).exp()
    clipped = ((A > 0) & (r > 1 + CLIP)) | ((A < 0) & (r < 1 - CLIP))
    term = -torch.minimum(r * A, r.clamp(1 - CLIP, 1 + CLIP) * A)
    dterm = torch.where(clipped, 0.0, -A * r)
    kl = torch.zeros_like(r)
    if s["ref"] is not None:
        d = s["ref"] - logp
        kl = d.expm1() - d
        term = term + KL * kl
        dterm = dterm - KL * d.expm1()
    zero = torch.zeros_like(w)
    c = torch.where(w != 0, w * dterm, zero)
    total = [torch.where(w != 0, w * v, zero).sum() for v in (term, kl, clipped.float())]
    return {"loss": total[0], "kl": total[1], "clipped": total[2], "logprobs": logp,
            "grad": _grad(p, s["targets"], c, s["logits"].dtype)}


def _plain_preference(s):
    w, off, T = s["weights"], s["offsets"], len(s["weights"])
    logp, p = _rows(s["logits"], s["targets"])
    logp = torch.where(w != 0, logp, 0.0)
    gain = torch.where(w != 0, w * (logp - s["ref"]), 0.0)
    t = torch.arange(T, device=w.device)
    member = ((t >= off[:-1, None]) & (t < off[1:, None])).float()
    sums = (member * gain).sum(1)
    z = BETA * (sums[0::2] - sums[1::2])
    pairs = len(z)
    loss = (torch.relu(-z) + (-z.abs()).exp().log1p()).sum() / pairs
    dz = -1.0 / (1.0 + z.exp()) / pairs
    side = BETA * torch.stack([dz, -dz], 1).reshape(-1)
    c = w * (member * side[:, None]).sum(0)
    return {"loss": loss, "margins": z, "logprobs": logp, "grad": _grad(p, s["targets"], c, s["logits"].dtype)}


def _plain_clip(s):
    g = s["grads"].float()
    norm = g.square().sum().sqrt()
    coef = (MAX_NORM / (norm + EPS)).clamp(max=1.0)
    s["out"].copy_(g * coef)
    return {"norm": norm, "out": s["out"]}


def _own(s):
    from allreduce_reduction_emulated_gb300 import losses

    op = s["case"]["op"]
    if op == "logprobs":
        return losses.token_logprobs(s["logits"], s["targets"])
    if op == "policy":
        r = losses.policy_loss(s["logits"], s["targets"], s["old"], s["advantages"], ref_logprobs=s["ref"],
                               weights=s["weights"], clip_low=CLIP, clip_high=CLIP,
                               kl_coef=KL if s["ref"] is not None else 0.0)
        return {"loss": r.loss, "kl": r.kl, "clipped": r.clipped, "logprobs": r.logprobs, "grad": r.grad}
    if op == "preference":
        r = losses.preference_loss(s["logits"], s["targets"], s["offsets"], s["ref"], weights=s["weights"], beta=BETA)
        return {"loss": r.loss, "margins": r.margins, "logprobs": r.logprobs, "grad": r.grad}
    return {"norm": s["clipper"].clip(MAX_NORM), "out": s["out"]}


_PLAIN = {"logprobs": _plain_logprobs, "policy": _plain_policy, "preference": _plain_preference, "clip": _plain_clip}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    es = ES[case["dtype"]]
    if case["op"] == "clip":
        return {"bytes": 2 * es * case["total"], "flops": 3 * case["total"]}
    T, V = _tokens(case), case["vocab"]
    read = T - _masked(case)                         # a masked row's logits are not needed
    if case["op"] == "logprobs":
        return {"bytes": T * V * es + T * (8 + 4), "flops": 4 * T * V}
    per_token = 8 + 4 * (4 + bool(case["kl"])) if case["op"] == "policy" else 8 + 4 * 3
    return {"bytes": (read + T) * V * es + T * per_token, "flops": 6 * read * V}


# ------------------------------------------------------------------ 64 bits

def _logp_and_grad(logits, targets, rows, c=None):
    """log_softmax at the targets of some rows in 64 bits and, with c, the gradient of sum(c * logp)."""
    x = logits[rows].double().requires_grad_(c is not None)
    logp = torch.log_softmax(x, 1)[torch.arange(x.shape[0], device=x.device), targets[rows]]
    if c is None:
        return logp, None
    return logp.detach(), torch.autograd.grad(logp, x, c[rows])[0]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        g = s["grads"]
        parts = g.split(1 << 27)
        norm = sum(torch.linalg.vector_norm(p.double()) ** 2 for p in parts) ** 0.5
        coef = min(1.0, MAX_NORM / (norm.item() + EPS))
        return {"norm": norm, "out": torch.cat([p.double() * coef for p in parts])}
    logits, targets = s["logits"], s["targets"]
    T = len(targets)
    step = max(1, (1 << 27) // logits.shape[1])
    spans = [slice(a, min(T, a + step)) for a in range(0, T, step)]
    logp = torch.cat([_logp_and_grad(logits, targets, r)[0] for r in spans])
    if case["op"] == "logprobs":
        return logp
    w = s["weights"].double()
    alive = w > 0
    logp[~alive] = 0.0
    v = logp.clone().requires_grad_()
    if case["op"] == "policy":
        ratio = torch.exp(v[alive] - s["old"].double()[alive])
        A = s["advantages"].double()[alive]
        bounded = torch.where(A >= 0, ratio.clamp(max=1 + CLIP), ratio.clamp(min=1 - CLIP))
        kl = torch.zeros_like(ratio)
        if s["ref"] is not None:
            q = s["ref"].double()[alive] - v[alive]
            kl = torch.expm1(q) - q
        loss = (w[alive] * (KL * kl - A * bounded)).sum()
        out = {"loss": loss.detach(), "kl": (w[alive] * kl).sum().detach(),
               "clipped": (w[alive] * (bounded != ratio)).sum().detach()}
    else:
        gain = torch.where(alive, w * (v - s["ref"].double()), 0.0)
        off = s["offsets"].tolist()
        sums = torch.stack([gain[a:b].sum() for a, b in zip(off, off[1:])])
        z = BETA * (sums[0::2] - sums[1::2])
        loss = -torch.nn.functional.logsigmoid(z).mean()
        out = {"loss": loss.detach(), "margins": z.detach()}
    c = torch.autograd.grad(loss, v)[0]
    grad = torch.empty(logits.shape, dtype=torch.float64, device="cuda")
    for r in spans:
        grad[r] = _logp_and_grad(logits, targets, r, c)[1]
    return {**out, "logprobs": logp, "grad": grad}
