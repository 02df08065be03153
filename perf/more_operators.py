"""More operators of the data-parallel training step, and what is measured of them.

Before the all-reduce: the products of layers whose weights are chosen by expert, and their
gradients.  Rows are sorted by expert; expert e has rows [offsets[e], offsets[e + 1]), as many as
the router gave it, and rows behind the last one belong to nobody.  After clipping: the update made
of the reduced gradients, orthogonalised by Newton-Schulz products.

    op = "product"      y[t] = W_e x[t]
    op = "gradients"    dx[t] = W_e^T dy[t],  dW_e = sum over e's rows of dy[t] x[t]^T
    op = "orthogonal"   momentum, and the orthogonalised update of stacks of matrices

own = False runs plain torch operations in 32 bits; own = True the package's operators.
"""
import math
import random

import torch

own = False

BETA = 0.95                                # orthogonal: momentum
STEPS = 5                                  # orthogonal: Newton-Schulz steps, and the usual coefficients of a step
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
ES = {"float32": 4, "bfloat16": 2}
# the weight matrices of a layer of the 1.2B-parameter gradient workload
LAYER = ((2048, 8192), (8192, 2048), (2048, 6144), (2048, 2048))


def listed():
    return [
        # a few tokens of a small model: latency
        {"name": "product 5x4 512-1024", "op": "product", "rows": 5, "experts": 4, "in": 512, "out": 1024, "skew": 0.5,
         "tail": 0, "layout": "out_in", "dtype": "bfloat16"},
        # eight sampled tokens, two experts each: every expert's weights are read for a row or two
        {"name": "product 16x8 2048-8192", "op": "product", "rows": 16, "experts": 8, "in": 2048, "out": 8192,
         "skew": 0.5, "tail": 0, "layout": "out_in", "dtype": "bfloat16"},
        # an ordinary micro-batch
        {"name": "product 4096x8 2048-8192", "op": "product", "rows": 4096, "experts": 8, "in": 2048, "out": 8192,
         "skew": 0.5, "tail": 0, "layout": "out_in", "dtype": "bfloat16"},
        # many small experts, weights with the outputs next to each other, a batch padded to its capacity
        {"name": "product 16384x64 2048-1024", "op": "product", "rows": 16384, "experts": 64, "in": 2048, "out": 1024,
         "skew": 1.0, "tail": 500, "layout": "in_out", "dtype": "bfloat16"},
        # odd sizes, at which no row starts at a whole vector; 32-bit results
        {"name": "product 1000x7 1001-1431 f32", "op": "product", "rows": 1000, "experts": 7, "in": 1001, "out": 1431,
         "skew": 1.0, "tail": 3, "layout": "out_in", "dtype": "float32"},
        # the backward pass of a short answer
        {"name": "gradients 64x8 2048-2048", "op": "gradients", "rows": 64, "experts": 8, "in": 2048, "out": 2048,
         "skew": 1.0, "tail": 0, "layout": "out_in", "dtype": "bfloat16"},
        # an ordinary micro-batch; the gradients go into 32-bit buckets
        {"name": "gradients 4096x8 8192-2048 f32", "op": "gradients", "rows": 4096, "experts": 8, "in": 8192,
         "out": 2048, "skew": 0.5, "tail": 0, "layout": "out_in", "dtype": "float32"},
        # a large one
        {"name": "gradients 16384x16 2048-8192", "op": "gradients", "rows": 16384, "experts": 16, "in": 2048,
         "out": 8192, "skew": 1.0, "tail": 100, "layout": "out_in", "dtype": "bfloat16"},
        # one small matrix: latency
        {"name": "orthogonal 256x256", "op": "orthogonal", "stacks": "1x256x256", "dtype": "bfloat16",
         "momentum": False},
        # the layers of a small model: several shapes, a tall one among them, odd sizes
        {"name": "orthogonal 30 small f32", "op": "orthogonal", "stacks": "8x128x512+8x512x128+12x128x128+1x96x1000+1x65x97",
         "dtype": "float32", "momentum": True},
        # a layer's experts
        {"name": "orthogonal 16x1024x2048", "op": "orthogonal", "stacks": "16x1024x2048", "dtype": "bfloat16",
         "momentum": True},
        # two layers of the 1.2B-parameter gradient workload
        {"name": "orthogonal 2 layers f32", "op": "orthogonal", "stacks": "+".join("2x%dx%d" % s for s in LAYER),
         "dtype": "float32", "momentum": True},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _side(rng, lo, hi):
    """A side of a matrix: mostly whole tiles, some whole vectors, some odd."""
    n = _log_between(rng, lo, hi)
    kind = rng.random()
    unit = 128 if kind < 0.45 else 8 if kind < 0.8 else 1
    return max(lo, -(-n // unit) * unit)


def draw(rng):
    op = rng.choice(["product", "gradients", "orthogonal"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    if op == "orthogonal":
        left = _flops_of("+".join("2x%dx%d" % s for s in LAYER))
        stacks = []
        for _ in range(rng.randint(1, 4)):
            m, n = _side(rng, 16, 4096), _side(rng, 16, 8192)
            if rng.random() < 0.4:
                m, n = n, m
            one = _flops_of("1x%dx%d" % (m, n))
            count = min(_log_between(rng, 1, 32), int(left // one))
            if count:
                stacks.append("%dx%dx%d" % (count, m, n))
                left -= count * one
        return {"op": op, "stacks": "+".join(stacks) or "1x100x200", "dtype": dtype, "momentum": rng.random() < 0.6}
    experts, fan_in, fan_out = _log_between(rng, 1, 64), _side(rng, 64, 8192), _side(rng, 64, 8192)
    experts = max(1, min(experts, (1 << 28) // (fan_in * fan_out)))
    rows = _log_between(rng, 1, 16384)
    rows = max(1, min(rows, 16384 * 2048 * 8192 // (fan_in * fan_out), (1 << 28) // (fan_in + fan_out)))
    return {"op": op, "rows": rows, "experts": experts, "in": fan_in, "out": fan_out,
            "skew": rng.choice([0.0, 0.5, 1.0]), "tail": rng.choice([0, 0, rng.randint(1, 1 + rows // 16)]),
            "layout": rng.choice(["out_in", "out_in", "in_out"]), "dtype": dtype}


# ------------------------------------------------------------------ inputs

def _counts(case):
    """Rows of each expert, the same for every seed: the router's choices are uneven, and where rows
    are few some experts have none."""
    r = random.Random(case["rows"] * 1_000_003 + case["experts"])
    load = [r.uniform(1.0 - 0.6 * case["skew"], 1.0 + case["skew"]) for _ in range(case["experts"])]
    at = [int(case["rows"] * sum(load[:e]) / sum(load)) for e in range(case["experts"])] + [case["rows"]]
    return [b - a for a, b in zip(at, at[1:])]


def _stacks(case_or_text):
    text = case_or_text if isinstance(case_or_text, str) else case_or_text["stacks"]
    return [tuple(int(v) for v in s.split("x")) for s in text.split("+")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = getattr(torch, case["dtype"])

    def normal(shape, sigma, kind):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, sigma, generator=gen).to(kind)

    if case["op"] == "orthogonal":
        grads, momentum = [], []
        for count, m, n in _stacks(case):
            # a few strong directions over the noise of a batch
            u, v = normal((count, m, 4), 1.0, torch.float32), normal((count, 4, n), 1.0, torch.float32)
            noise = normal((count, m, n), 1e-3, torch.float32)
            grads.append(noise.add_(torch.bmm(u, v), alpha=2e-4).to(dtype))
            if case["momentum"]:
                momentum.append(normal((count, m, n), 3e-3, torch.float32))
        state = {"case": case, "grads": grads, "momentum": momentum}
        if own:
            from allreduce_reduction_emulated_gb300.orthogonal import Orthogonalizer
            state["handle"] = Orthogonalizer(grads, momentum=momentum or None, beta=BETA, steps=STEPS,
                                             coefficients=COEFFICIENTS, eps=EPS)
        return state
    E, K, N, T = case["experts"], case["in"], case["out"], case["rows"] + case["tail"]
    weights = (normal((E, N, K), K ** -0.5, torch.bfloat16) if case["layout"] == "out_in"
               else normal((E, K, N), K ** -0.5, torch.bfloat16).transpose(1, 2))
    n = torch.tensor(_counts(case), device="cuda")
    state = {"case": case, "weights": weights, "x": normal((T, K), 1.0, torch.bfloat16),
             "offsets": torch.cat([n.new_zeros(1), n.cumsum(0)]), "most": max(_counts(case))}
    if case["op"] == "gradients":
        state["dy"] = normal((T, N), 1e-2, torch.bfloat16)
    return state


# ------------------------------------------------------------------ the plain forms

def _slots(s):
    """Each row's place among experts that all have as many rows as the fullest one."""
    off, most = s["offsets"], s["most"]
    t = torch.arange(s["case"]["rows"], device=off.device)
    e = torch.searchsorted(off, t, right=True) - 1
    return e * most + t - off[e]


def _padded(s, x, slots):
    """(experts, most, columns) in 32 bits, zeros where an expert has fewer rows."""
    E = s["case"]["experts"]
    wide = torch.zeros(E * s["most"], x.shape[1], device=x.device)
    wide[slots] = x[:len(slots)].float()
    return wide.view(E, s["most"], x.shape[1])


def _rows(wide, slots, rows, dtype):
    """The rows back in their order; zeros for those of no expert."""
    out = torch.zeros(rows, wide.shape[2], dtype=dtype, device=wide.device)
    out[:len(slots)] = wide.reshape(-1, wide.shape[2])[slots].to(dtype)
    return out


def _plain_product(s):
    slots = _slots(s)
    y = torch.bmm(_padded(s, s["x"], slots), s["weights"].float().transpose(1, 2))
    return _rows(y, slots, len(s["x"]), getattr(torch, s["case"]["dtype"]))


def _plain_gradients(s):
    slots = _slots(s)
    dy, x = _padded(s, s["dy"], slots), _padded(s, s["x"], slots)
    dx = torch.bmm(dy, s["weights"].float())
    dw = torch.bmm(dy.transpose(1, 2), x)
    return {"dx": _rows(dx, slots, len(s["x"]), torch.bfloat16), "dw": dw.to(getattr(torch, s["case"]["dtype"]))}


def _plain_update(g, momentum):
    u = g.float()
    if momentum is not None:
        momentum.mul_(BETA).add_(u)
        u = u + BETA * momentum
    tall = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2) if tall else u
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        s = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * s + c * torch.bmm(s, s), x)
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16)


def _plain_orthogonal(s):
    momentum = s["momentum"] or [None] * len(s["grads"])
    return {"updates": [_plain_update(g, m) for g, m in zip(s["grads"], momentum)], "momentum": s["momentum"]}


def _own(s):
    case = s["case"]
    if case["op"] == "orthogonal":
        return {"updates": s["handle"].update(), "momentum": s["momentum"]}
    from allreduce_reduction_emulated_gb300 import experts

    dtype = getattr(torch, case["dtype"])
    if case["op"] == "product":
        return experts.expert_product(s["x"], s["weights"], s["offsets"], dtype=dtype)
    dx, dw = experts.expert_gradients(s["dy"], s["x"], s["weights"], s["offsets"], dw_dtype=dtype)
    return {"dx": dx, "dw": dw}


_PLAIN = {"product": _plain_product, "gradients": _plain_gradients, "orthogonal": _plain_orthogonal}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def _flops_of(text):
    """Of a step: s s^T and its square are symmetric (half of each suffices), the product with x is whole."""
    total = 0
    for count, m, n in _stacks(text):
        s, l = min(m, n), max(m, n)
        total += count * STEPS * (3 * s * s * l + s ** 3)
    return total


def work(case):
    if case["op"] == "orthogonal":
        n = sum(count * m * k for count, m, k in _stacks(case))
        return {"bytes": n * (ES[case["dtype"]] + 2 + (8 if case["momentum"] else 0)), "flops": _flops_of(case["stacks"])}
    K, N, R, T = case["in"], case["out"], case["rows"], case["rows"] + case["tail"]
    used = sum(c > 0 for c in _counts(case))
    if case["op"] == "product":
        return {"bytes": 2 * (R * K + used * K * N) + ES[case["dtype"]] * T * N, "flops": 2 * R * K * N}
    return {"bytes": 2 * (R * (K + N) + used * K * N + T * K) + ES[case["dtype"]] * case["experts"] * K * N,
            "flops": 4 * R * K * N}


# ------------------------------------------------------------------ 64 bits

def _exact_update(g, momentum):
    u = g.double()
    if momentum is not None:
        momentum = BETA * momentum.double() + u
        u = u + BETA * momentum
    a, b, c = COEFFICIENTS
    wide = u if u.shape[0] <= u.shape[1] else u.t()
    x = wide / (torch.linalg.matrix_norm(wide) + EPS)
    one = torch.eye(len(x), dtype=x.dtype, device=x.device)
    for _ in range(STEPS):
        s = x @ x.t()
        x = (a * one + s @ (b * one + c * s)) @ x
    return (x if wide is u else x.t()), momentum


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orthogonal":
        got = {"updates": [], "momentum": []}
        for k, g in enumerate(s["grads"]):
            parts = [_exact_update(x, s["momentum"][k][i] if s["momentum"] else None) for i, x in enumerate(g)]
            got["updates"].append(torch.stack([p[0] for p in parts]))
            if s["momentum"]:
                got["momentum"].append(torch.stack([p[1] for p in parts]))
        return got
    off = s["offsets"].tolist()
    x, w = s["x"], s["weights"]
    spans = [(e, slice(a, b)) for e, (a, b) in enumerate(zip(off, off[1:]))]
    if case["op"] == "product":
        y = torch.zeros(len(x), case["out"], dtype=torch.float64, device="cuda")
        for e, r in spans:
            y[r] = torch.einsum("tk,nk->tn", x[r].double(), w[e].double())
        return y
    dx = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(w.shape, dtype=torch.float64, device="cuda")
    for e, r in spans:
        dx[r] = torch.einsum("tn,nk->tk", s["dy"][r].double(), w[e].double())
        dw[e] = torch.einsum("tn,tk->nk", s["dy"][r].double(), x[r].double())
    return {"dx": dx, "dw": dw}
