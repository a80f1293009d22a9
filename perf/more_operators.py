"""Cases and plain forms of the operators at the experts' two ends: the router with the balance loss
(forward and gradients), the weighted combine with its gradients, and low-rank adapters of many
requests beside a shared projection.

`run` computes a case in elementary torch operations (32 bits inside, 64 for selection scores with a
bias and for the loss's long sums, rounded once at the end), or with `own` set through this package's
entry points on the same inputs.

A token is `live` where its entry is not negative (padding behind it); a slot is (token, choice).
Adapters are grouped by the align over the rows' adapter ids, which a program makes once a step and
keeps for every projection, so `prepare` makes it.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
BALANCE = 0.01   # the loss's share in a training step's objective


# ----------------------------------------------------------------------------- cases
def _router(M, E, k, dtype, score, bias, renorm, pad, masked=0):
    return {"M": M, "experts": E, "top_k": k, "dtype": dtype, "score": score, "bias": bias, "renorm": renorm,
            "scale": 1.0 if score == "softmax" else 2.5, "pad": pad, "masked": masked}


def _combine(M, k, H, live, norm):
    return {"op": "combine", "M": M, "top_k": k, "H": H, "live": live, "norm": norm}


def _adapters(M, N, K, r, n, none, ragged, scales, block_m):
    return {"op": "adapters", "M": M, "N": N, "K": K, "rank": r, "adapters": n, "none": none, "ragged": ragged,
            "scales": scales, "block_m": block_m}


def listed():
    return [
        # the router of a decode step: one token of one request (latency)
        {"name": "route_tokens1_e256_k8", "op": "route", **_router(1, 256, 8, "fp32", "sigmoid", True, True, 0.0)},
        # a decode batch on 128 experts whose weights are a softmax over the chosen logits
        {"name": "route_tokens64_e128_k4", "op": "route", **_router(64, 128, 4, "bf16", "softmax", False, True, 0.0)},
        # a large prefill batch, sigmoid scores with a selection bias
        {"name": "route_tokens32768_e256_k8", "op": "route", **_router(32768, 256, 8, "bf16", "sigmoid", True, True, 0.0)},
        # a training step's router with counts, balance loss and the gradient of the logits: few experts, a whole
        # slice's batch, and padded fp32 logits with switched-off experts and an odd number of each
        {"name": "balance_tokens2304_e8_k2", "op": "balance", **_router(2304, 8, 2, "bf16", "softmax", False, False, 0.0)},
        {"name": "balance_tokens4096_e256_k8", "op": "balance", **_router(4096, 256, 8, "bf16", "sigmoid", True, True, 0.0)},
        {"name": "balance_tokens32765_e129_k4", "op": "balance",
         **_router(32765, 129, 4, "fp32", "softmax", False, True, 0.2, masked=3)},
        # the combine of a training step with its gradients: two choices of 8 local experts, a normed combine with odd
        # numbers of tokens and columns, and one GPU's slice of a batch of 8 choices each
        {"name": "combine_tokens2304_k2_h512", **_combine(2304, 2, 512, 1.0, False)},
        {"name": "combine_norm_tokens509_k4_h2880", **_combine(509, 4, 2880, 1.0, True)},
        {"name": "combine_norm_tokens4096_k8_h4096", **_combine(4096, 8, 4096, 0.71, True)},
        # adapters: a decode step of one request, a decode batch in which nearly every request has its own, and a
        # prefill batch of a few long requests with adapters of several ranks, some rows without one
        {"name": "adapters_tokens1_r16", **_adapters(1, 4096, 7168, 16, 8, 0.0, False, True, 16)},
        {"name": "adapters_tokens64_r16_many", **_adapters(64, 8192, 4096, 16, 64, 0.1, False, True, 16)},
        {"name": "adapters_tokens8179_r64", **_adapters(8179, 4096, 4096, 64, 6, 0.15, True, True, 64)},
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step)


def draw(rng):
    op = rng.choice(["route", "balance", "combine", "adapters"])
    if op in ("route", "balance"):
        E = rng.choice([8, 16, 60, 64, 128, 129, 160, 256, 384, 512])
        k = rng.randint(1, min(8, E))
        M = max(1, _log_int(rng, 1, 32765) * 129 // max(129, E))
        return {"op": op, **_router(M, E, k, rng.choice(["bf16", "fp32"]), rng.choice(["softmax", "sigmoid"]),
                                    rng.random() < 0.5, rng.random() < 0.5, rng.choice([0.0, 0.0, 0.3]),
                                    rng.choice([0, 0, min(3, E - k)]))}
    if op == "combine":
        k, H = rng.randint(1, 8), 8 * rng.randint(32, 512)
        return _combine(_log_int(rng, 1, 4096), k, H, rng.choice([1.0, 0.71, 0.13]), rng.random() < 0.5)
    M, n = _log_int(rng, 1, 8179), _log_int(rng, 1, 64)
    per = M / min(M, n)
    return _adapters(M, 8 * rng.randint(16, 512), 8 * rng.randint(16, 512), rng.choice([8, 16, 24, 32, 64]), n,
                     rng.choice([0.0, 0.15, 0.5]), rng.random() < 0.5, rng.random() < 0.7,
                     16 if per <= 16 else 32 if per <= 32 else 64)


# ----------------------------------------------------------------------------- inputs
def _generator(seed, what):
    return torch.Generator(device="cuda").manual_seed(seed * 32 + what)


def _normal(shape, seed, what):
    return torch.randn(shape, device="cuda", generator=_generator(seed, what))


def _uniform(shape, seed, what):
    return torch.rand(shape, device="cuda", generator=_generator(seed, what))


def _prepare_router(case, seed):
    """Logits about as wide as a trained router's, some experts more popular than others."""
    M, E, k = case["M"], case["experts"], case["top_k"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    x = 1.2 * _normal((M, E), seed, 1) + 0.6 * _normal((E,), seed, 2)
    if case["masked"]:
        x[:, torch.argsort(_uniform((E,), seed, 3))[: case["masked"]]] = -math.inf   # experts switched off
    st = {"logits": x.to(dtype), "bias": 0.05 * _normal((E,), seed, 4) if case["bias"] else None, "live": None}
    if case["pad"]:   # the tail of each row of 64 tokens is padding
        at = torch.arange(M, device="cuda") % 64
        length = 64 * (1.0 - 2.0 * case["pad"] * _uniform((M // 64 + 1,), seed, 5).repeat_interleave(64)[:M])
        st["live"] = torch.where(at < length, 0, -1).to(torch.int32)
    if case["op"] == "balance":
        st["grad"] = _normal((M, k), seed, 6) / M
        st["share"] = torch.full((), BALANCE, device="cuda")
    else:
        st["ids"] = torch.empty((M, k), dtype=torch.int32, device="cuda")
        st["weights"] = torch.empty((M, k), device="cuda")
    return st


def _prepare_combine(case, seed):
    M, k, H = case["M"], case["top_k"], case["H"]
    y = torch.empty((M * k, H), dtype=torch.bfloat16, device="cuda")
    gen = _generator(seed, 7)
    for r in range(0, M * k, 8192):
        y[r: r + 8192] = torch.randn((min(8192, M * k - r), H), device="cuda", generator=gen).bfloat16()
    g = torch.softmax(_normal((M, k), seed, 8), dim=-1)
    live = _uniform((M, k), seed, 9) < case["live"]
    st = {"y": y, "weights": g, "local": torch.where(live, 0, -1).to(torch.int32),
          "norm": (1.0 + 0.2 * _normal((H,), seed, 10)).bfloat16() if case["norm"] else None,
          "grad": _normal((M, H), seed, 11).bfloat16()}
    y[st["local"].view(-1) < 0] = 0.0     # what the down product leaves in rows of dropped slots
    return st


def _adapter_ids(case, seed):
    """The adapter of every row: runs of rows for long requests, one row each in a decode batch."""
    M, n = case["M"], case["adapters"]
    r = np.random.default_rng([seed, 1])
    requests = min(M, 2 * n)
    cuts = np.sort(r.choice(M - 1, size=requests - 1, replace=False) + 1) if requests > 1 else np.zeros(0, np.int64)
    which = r.permutation(np.arange(requests) % n)
    which[r.random(requests) < case["none"]] = -1
    return np.repeat(which, np.diff(np.concatenate([[0], cuts, [M]]))).astype(np.int32)


def _prepare_adapters(case, seed):
    M, N, K, r, n, B = (case[key] for key in ("M", "N", "K", "rank", "adapters", "block_m"))
    ids = _adapter_ids(case, seed)
    order = np.argsort(ids, kind="stable").astype(np.int32)
    order = order[ids[order] >= 0]
    counts = np.bincount(ids[order], minlength=n)
    blocks = -(-counts // B)
    most = -(-(M + min(n, M) * (B - 1)) // B)
    sorted_ids, block_ids, at, seen = np.full(most * B, M, np.int32), np.full(most, -1, np.int32), 0, 0
    for a in range(n):
        sorted_ids[at * B: at * B + counts[a]] = order[seen: seen + counts[a]]
        block_ids[at: at + blocks[a]] = a
        at, seen = at + blocks[a], seen + counts[a]
    dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    ranks = None
    if case["ragged"]:
        ranks = np.random.default_rng([seed, 2]).choice([max(1, r // 8), max(1, r // 2), r], size=n).astype(np.int32)
    return {"x": _normal((M, K), seed, 12).bfloat16(), "base": _normal((M, N), seed, 13).bfloat16(),
            "A": (_normal((n, r, K), seed, 14) / math.sqrt(K)).bfloat16(),
            "B": (_normal((n, N, r), seed, 15) / math.sqrt(r)).bfloat16(),
            "scales": 0.25 + _uniform((n,), seed, 16) if case["scales"] else None, "ranks": None if ranks is None else dev(ranks),
            "rank_list": [r] * n if ranks is None else [int(v) for v in ranks],
            "align": (dev(sorted_ids), dev(block_ids), dev(np.array([at * B], np.int32)), dev(ids.reshape(M, 1))),
            "rows": {a: dev(np.flatnonzero(ids == a)) for a in range(n) if counts[a]},
            "out": torch.empty((M, N), dtype=torch.bfloat16, device="cuda")}


def prepare(case, seed):
    if case["op"] in ("route", "balance"):
        st = _prepare_router(case, seed)
    elif case["op"] == "combine":
        st = _prepare_combine(case, seed)
    else:
        st = _prepare_adapters(case, seed)
    st["case"] = case
    return st


# ----------------------------------------------------------------------------- plain forms
def _scores(x, score):
    """The experts' scores, and their probabilities (which sum to one in a row), of logits x (fp32 or fp64)."""
    if score == "softmax":
        top = x.amax(dim=-1, keepdim=True)
        e = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
        p = e / e.sum(dim=-1, keepdim=True)
        return p, p
    s = 1.0 / (1.0 + torch.exp(-x))
    return s, s / s.sum(dim=-1, keepdim=True)


def _select(st):
    """ids int32 [M, k] (-1: none) and the chosen slots [M, k]."""
    case, x = st["case"], st["logits"].float()
    key = x
    if st["bias"] is not None:
        key = _scores(x.double(), case["score"])[0] + st["bias"].double()
    key = torch.where(x > -math.inf, key, -math.inf)
    key, order = torch.sort(key, dim=-1, descending=True, stable=True)
    order, chosen = order[:, : case["top_k"]], key[:, : case["top_k"]] > -math.inf
    if st["live"] is not None:
        chosen = chosen & (st["live"] >= 0)[:, None]
    return torch.where(chosen, order, -1).to(torch.int32), chosen


def _plain_route(st):
    case = st["case"]
    ids, chosen = _select(st)
    scores, _ = _scores(st["logits"].float(), case["score"])
    picked = torch.where(chosen, torch.gather(scores, 1, ids.clamp_min(0).long()), 0.0)
    if case["renorm"]:
        picked = picked / picked.sum(dim=-1, keepdim=True).clamp_min(1e-30)
    return [ids, picked * case["scale"]], chosen


def _plain_balance(st):
    case, k, E = st["case"], st["case"]["top_k"], st["case"]["experts"]
    (ids, weights), chosen = _plain_route(st)
    x, at = st["logits"].float(), ids.clamp_min(0).long()
    s, q = _scores(x, case["score"])
    live = torch.ones(x.shape[0], device=x.device) if st["live"] is None else (st["live"] >= 0).float()
    tokens = live.sum().clamp_min(1.0)
    counts = torch.zeros(E + 1, dtype=torch.int32, device=x.device)
    counts.index_add_(0, torch.where(chosen, ids, E).view(-1).long(), torch.ones(ids.numel(), dtype=torch.int32, device=x.device))
    counts = counts[:E]
    share = counts.double() / counts.sum().clamp_min(1)
    means = (q * live[:, None]).double().sum(dim=0) / tokens.double()
    loss = E * (share * means).sum()
    # gradients: of the weights, then of the loss
    c, grad = case["scale"], st["grad"]
    h = weights / c
    slope = 1.0 if case["score"] == "softmax" else 1.0 - torch.gather(s, 1, at)
    if case["renorm"]:
        d = c * h * slope * (grad - (grad * h).sum(dim=-1, keepdim=True))
    elif case["score"] == "softmax":
        d = c * h * grad
    else:
        d = c * h * slope * grad
    a = st["share"] * E * share.float() / tokens
    out = q * (a - (a * q).sum(dim=-1, keepdim=True))
    if case["score"] == "sigmoid":
        out = out * (1.0 - s)
    elif not case["renorm"]:
        out = out - c * q * (grad * h).sum(dim=-1, keepdim=True)
    out = out.scatter_add(1, at, torch.where(chosen, d, 0.0)) * live[:, None]
    return [ids, weights, counts, loss.float(), out.to(st["logits"].dtype)]


def _plain_combine(st):
    case = st["case"]
    M, k, H = case["M"], case["top_k"], case["H"]
    live = (st["local"] >= 0).float()
    y, grad = st["y"].float().view(M, k, H), st["grad"].float()[:, None, :]
    g = st["weights"] * live
    if st["norm"] is None:
        out = (g[..., None] * y).sum(dim=1)
        return [out.bfloat16(), (g[..., None] * grad).view(M * k, H).bfloat16(), (grad * y).sum(dim=-1) * live]
    n = st["norm"].float()
    z = y * n
    r = 1.0 / torch.sqrt((z * z).mean(dim=-1) + EPS)
    out = ((g * r)[..., None] * z).sum(dim=1)
    d = (grad * z).sum(dim=-1)
    dz = (g * r)[..., None] * (grad - (r * r * d / H)[..., None] * z)
    return [out.bfloat16(), (dz * n).view(M * k, H).bfloat16(), r * d * live, (dz * y).sum(dim=(0, 1)).bfloat16()]


def _plain_adapters(st):
    out = st["base"].float()
    for a, rows in st["rows"].items():
        r = st["rank_list"][a]
        delta = (st["x"][rows].float() @ st["A"][a, :r].float().T) @ st["B"][a, :, :r].float().T
        out[rows] += delta if st["scales"] is None else delta * st["scales"][a]
    return [out.bfloat16()]


def run(state):
    st, case = state, state["case"]
    op = case["op"]
    if not own:
        if op == "route":
            return _plain_route(st)[0]
        return {"balance": _plain_balance, "combine": _plain_combine, "adapters": _plain_adapters}[op](st)
    import quantized_mixture_experts_align_amd as P
    if op in ("route", "balance"):
        how = dict(score=case["score"], bias=st["bias"], renormalise=case["renorm"], scale=case["scale"], live=st["live"])
        if op == "route":
            return list(P.moe_router(st["logits"], case["top_k"], out=(st["ids"], st["weights"]), **how))
        logits = st["logits"].detach().requires_grad_(True)
        r = P.moe_experts_router(logits, case["top_k"], **how)
        (d,) = torch.autograd.grad((r.weights, r.balance), logits, (st["grad"], st["share"]))
        return [r.ids, r.weights.detach(), r.counts, r.balance.detach(), d]
    if op == "combine":
        leaves = [t.detach().requires_grad_(True) for t in (st["y"], st["weights"], st["norm"]) if t is not None]
        out = P.moe_experts_combine(leaves[0], leaves[1], st["local"], norm_w=leaves[2] if len(leaves) > 2 else None, eps=EPS)
        return [out.detach(), *torch.autograd.grad(out, leaves, st["grad"])]
    return [P.moe_adapters_add(st["base"], st["x"], st["A"], st["B"], st["align"], case["block_m"], scales=st["scales"],
                               ranks=st["ranks"], out=st["out"])]


# ----------------------------------------------------------------------------- floors
def work(case):
    op = case["op"]
    if op in ("route", "balance"):
        M, E, k = case["M"], case["experts"], case["top_k"]
        size = 2 if case["dtype"] == "bf16" else 4
        live = M * (1.0 - case["pad"])
        forward = live * E * size + 8.0 * M * k + 4 * E * case["bias"] + 4 * M * bool(case["pad"])
        if op == "route":
            return {"bytes": forward, "flops": live * E * 6.0}
        return {"bytes": forward + 4.0 * M * k + 4 * E + 8 + M * E * size, "flops": live * E * 16.0}
    if op == "combine":
        M, k, H = case["M"], case["top_k"], case["H"]
        live = M * k * case["live"]
        return {"bytes": live * H * 2.0 + M * k * H * 2.0 + 2 * M * H * 2.0 + 12.0 * M * k + (4 * H if case["norm"] else 0),
                "flops": live * H * (12.0 if case["norm"] else 5.0)}
    M, N, K, r, n = (case[key] for key in ("M", "N", "K", "rank", "adapters"))
    share = (1.0 / 8 + 1.0 / 2 + 1.0) / 3 if case["ragged"] else 1.0
    rows = M * (1.0 - case["none"])
    used = min(M, n) * (1.0 - case["none"] ** (2 if M >= 2 * n else 1))   # adapters that some request has
    return {"bytes": rows * K * 2.0 + M * N * 4.0 + used * share * r * (K + N) * 2.0 + 8.0 * M,
            "flops": 2.0 * rows * r * share * (K + N)}


# ----------------------------------------------------------------------------- the definition, in 64 bits
def _exact_router(st):
    case, k, E = st["case"], st["case"]["top_k"], st["case"]["experts"]
    x = st["logits"].double()
    M, dev = x.shape[0], x.device
    live = torch.ones(M, dtype=torch.bool, device=dev) if st["live"] is None else st["live"] >= 0
    if case["score"] == "softmax":
        s = torch.exp(x - torch.logsumexp(x, dim=-1, keepdim=True))
        q = s
    else:
        s = torch.sigmoid(x)
        q = s / s.sum(dim=-1, keepdim=True)
    left = x.clone() if st["bias"] is None else s + st["bias"].double()
    left[torch.isneginf(x)] = -math.inf
    columns = torch.arange(E, device=dev)
    hot = torch.zeros((M, E), dtype=torch.bool, device=dev)
    ids = torch.full((M, k), -1, dtype=torch.int64, device=dev)
    for j in range(k):
        best = left.amax(dim=-1, keepdim=True)
        at = torch.where(left == best, columns, E).amin(dim=-1)
        good = (best[:, 0] > -math.inf) & live
        ids[:, j] = torch.where(good, at, -1)
        mark = columns == at[:, None]
        hot |= mark & good[:, None]
        left = torch.where(mark, -math.inf, left)
    masked = torch.where(hot, s, 0.0)
    total = masked.sum(dim=-1, keepdim=True) if case["renorm"] else torch.ones((M, 1), dtype=torch.float64, device=dev)
    dense = torch.where(hot, case["scale"] * s / total, 0.0)
    weights = torch.where(ids >= 0, torch.gather(dense, 1, ids.clamp_min(0)), 0.0)
    if case["op"] == "route":
        return [ids.to(torch.int32), weights]
    # gradients through the Jacobians of each step: weights -> scores -> logits
    count = hot.sum(dim=0)
    tokens = max(1, int(live.sum()))
    f = count.double() / max(1, int(count.sum()))
    loss = E * (f * q[live].sum(dim=0)).sum() / tokens
    grad = torch.zeros((M, E), dtype=torch.float64, device=dev)
    grad.scatter_add_(1, ids.clamp_min(0), torch.where(ids >= 0, st["grad"].double(), 0.0))
    if case["renorm"]:    # d(c s / total) / ds
        ds = torch.where(hot, case["scale"] / total * (grad - (grad * masked).sum(dim=-1, keepdim=True) / total), 0.0)
    else:
        ds = case["scale"] * grad
    dq = (float(st["share"].double()) * E / tokens) * f[None, :].expand(M, E)
    if case["score"] == "softmax":
        ds = ds + dq
        dx = s * (ds - (ds * s).sum(dim=-1, keepdim=True))
    else:
        ds = ds + (dq - (dq * q).sum(dim=-1, keepdim=True)) / s.sum(dim=-1, keepdim=True)
        dx = ds * s * torch.sigmoid(-x)
    return [ids.to(torch.int32), weights, count.to(torch.int32), loss, torch.where(live[:, None], dx, 0.0)]


def _exact_combine(st):
    case = st["case"]
    M, k, H = case["M"], case["top_k"], case["H"]
    live = (st["local"] >= 0).double()
    out = torch.zeros((M, H), dtype=torch.float64, device="cuda")
    dy = torch.zeros((M, k, H), dtype=torch.float64, device="cuda")
    dg = torch.zeros((M, k), dtype=torch.float64, device="cuda")
    dn = torch.zeros(H, dtype=torch.float64, device="cuda")
    n = torch.ones(H, dtype=torch.float64, device="cuda") if st["norm"] is None else st["norm"].double()
    grad = st["grad"].double()
    for s in range(k):
        z = st["y"].view(M, k, H)[:, s].double() * n
        r = torch.ones(M, dtype=torch.float64, device="cuda")
        if st["norm"] is not None:
            r = (z.pow(2).sum(dim=-1) / H + EPS).rsqrt()
        unit = z * r[:, None]                                    # the normed row
        g = (st["weights"][:, s].double() * live[:, s])[:, None]
        out += g * unit
        dg[:, s] = (unit * grad).sum(dim=-1) * live[:, s]
        du = g * grad
        dz = du if st["norm"] is None else r[:, None] * (du - unit * (unit * du).sum(dim=-1, keepdim=True) / H)
        dy[:, s] = dz * n
        dn += (dz * st["y"].view(M, k, H)[:, s].double()).sum(dim=0)
    return [out, dy.view(M * k, H), dg] + ([] if st["norm"] is None else [dn])


def _exact_adapters(st):
    out = st["base"].double()
    owner = st["align"][3].view(-1)
    for a in range(st["A"].shape[0]):
        rows = torch.nonzero(owner == a).view(-1)
        if len(rows):
            r = st["rank_list"][a]
            inner = torch.mm(st["x"][rows].double(), st["A"][a, :r].double().t())
            gain = 1.0 if st["scales"] is None else st["scales"][a].double()
            out[rows] += torch.mm(inner * gain, st["B"][a, :, :r].double().t())
    return [out]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("route", "balance"):
        return _exact_router(st)
    return _exact_combine(st) if case["op"] == "combine" else _exact_adapters(st)
