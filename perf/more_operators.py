"""The operators of a policy update beyond the on-policy loss: losses over given log-probabilities (the clipped policy
loss with its KL term, the preference loss over pairs), the way back from the log-probabilities to the hidden states
and the head, and the gradients' global norm with clipping.

`run` computes each in its plain form, or with `own` through grpo_policy_loss_amd. Cases are plain dicts:

  op "logprobs": type, tokens, hidden, vocab, temperature, live (share of tokens whose gradient is not zero): the
                 log-probabilities of the targets, and the gradients of hidden states and head
  op "clip":     sequences, length, level of the ratio ("token", "sequence"), mean ("token", "sequence"), low, high, dual
                 (0: none), kl ("reverse", "forward"), beta (0: no reference), adv ("sequence", "token"): loss, statistics
                 and gradient
  op "pref":     pairs, length, kind ("sigmoid", "hinge", "square"), averaged (log ratios are means), reference,
                 smoothing, margin, nll: loss, rewards and gradient
  op "gradnorm": f32 and bf16, each "elements x count, ..." (empty: none), packed (tensors at odd offsets of one buffer,
                 or each on a 128-element boundary), norm ("l2", "max"), clip (the gradients scaled in place)
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
MAX_NORM = 1.0
PREF_BETA = 0.1


def listed():
    return [
        # a small float32 head: a launch's latency
        {"name": "logprobs tiny", "op": "logprobs", "type": "f32", "tokens": 512, "hidden": 256, "vocab": 1024, "temperature": 1.0, "live": 0.75},
        # a micro-batch of a 1.5B model: prompts and padding have no gradient
        {"name": "logprobs batch", "op": "logprobs", "type": "bf16", "tokens": 4096, "hidden": 1536, "vocab": 151936, "temperature": 1.0, "live": 0.7},
        # a micro-batch of an 8B model, sampled at a temperature, every token trained
        {"name": "logprobs long", "op": "logprobs", "type": "bf16", "tokens": 8192, "hidden": 4096, "vocab": 128256, "temperature": 0.9, "live": 1.0},
        # one micro-step of a second epoch over short completions: launches' latency
        {"name": "clip small", "op": "clip", "sequences": 8, "length": 64, "level": "token", "mean": "token", "low": 0.2, "high": 0.28, "dual": 0.0, "kl": "reverse", "beta": 0.04, "adv": "sequence"},
        # eight completions of a 20K context, a ratio for each token and the KL term
        {"name": "clip long", "op": "clip", "sequences": 8, "length": 20480, "level": "token", "mean": "token", "low": 0.2, "high": 0.28, "dual": 3.0, "kl": "reverse", "beta": 0.04, "adv": "sequence"},
        # a whole rollout batch at odd lengths, one ratio for each sequence
        {"name": "clip batch", "op": "clip", "sequences": 1021, "length": 16385, "level": "sequence", "mean": "sequence", "low": 0.0003, "high": 0.0004, "dual": 0.0, "kl": "reverse", "beta": 0.001, "adv": "sequence"},
        # one pair: launches' latency
        {"name": "pref pair", "op": "pref", "pairs": 1, "length": 513, "kind": "sigmoid", "averaged": False, "reference": True, "smoothing": 0.0, "margin": 0.0, "nll": 0.0},
        # a usual batch of pairs, with smoothed labels and the chosen one's likelihood
        {"name": "pref batch", "op": "pref", "pairs": 64, "length": 2048, "kind": "sigmoid", "averaged": False, "reference": True, "smoothing": 0.1, "margin": 0.0, "nll": 0.2},
        # many short pairs without a reference model, by their mean log-probabilities
        {"name": "pref many", "op": "pref", "pairs": 16384, "length": 511, "kind": "sigmoid", "averaged": True, "reference": False, "smoothing": 0.0, "margin": 0.5, "nll": 0.0},
        # two norm weights: launches' latency
        {"name": "gradnorm vectors", "op": "gradnorm", "f32": "1536x2", "bf16": "", "packed": False, "norm": "l2", "clip": False},
        # the matrices of a layer, bfloat16, beside float32 norm weights, clipped in place for an optimizer that takes no scale
        {"name": "gradnorm layer", "op": "gradnorm", "f32": "4096x2,257x3", "bf16": "16777216x4,100003x8", "packed": True, "norm": "l2", "clip": True},
        # the float32 gradient of a head, whose scale goes to the optimizer
        {"name": "gradnorm head", "op": "gradnorm", "f32": "233373696x1,1536x1", "bf16": "", "packed": False, "norm": "l2", "clip": False},
    ]


def _log(rng, low, high):
    """A whole number, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["logprobs", "clip", "pref", "gradnorm"])
    if op == "logprobs":
        kind = rng.choice(["f32", "bf16"])
        most = 8192 * 128256 * 4096 if kind == "bf16" else 1 << 36
        hidden = 8 * _log(rng, 8, 512)
        vocab = _log(rng, 2, 201088 if kind == "bf16" else 65537)
        return {"op": "logprobs", "type": kind, "tokens": _log(rng, 1, max(1, min(8192, most // (hidden * vocab)))), "hidden": hidden, "vocab": vocab,
                "temperature": rng.choice([1.0, round(rng.uniform(0.5, 1.5), 3)]), "live": round(rng.uniform(0.2, 1.0), 2)}
    if op == "clip":
        length = _log(rng, 1, 32768)
        level = rng.choice(["token", "sequence"])
        return {"op": "clip", "sequences": _log(rng, 1, max(1, min(8192, (1 << 24) // length))), "length": length, "level": level, "mean": rng.choice(["token", "sequence"]),
                "low": round(rng.uniform(0.05, 0.3), 3) if level == "token" else round(rng.uniform(1e-3, 0.05), 4), "high": round(rng.uniform(0.05, 0.4), 3) if level == "token" else round(rng.uniform(1e-3, 0.05), 4),
                "dual": rng.choice([0.0, round(rng.uniform(1.5, 4.0), 2)]), "kl": rng.choice(["reverse", "forward"]), "beta": rng.choice([0.0, round(rng.uniform(0.001, 0.1), 4)]),
                "adv": rng.choice(["sequence", "token"]) if level == "token" else "sequence"}
    if op == "pref":
        length = _log(rng, 1, 32768)
        kind = rng.choice(["sigmoid", "hinge", "square"])
        return {"op": "pref", "pairs": _log(rng, 1, max(1, min(16384, (1 << 23) // length))), "length": length, "kind": kind, "averaged": rng.random() < 0.5, "reference": rng.random() < 0.7,
                "smoothing": round(rng.uniform(0.0, 0.3), 3) if kind == "sigmoid" else 0.0, "margin": rng.choice([0.0, round(rng.uniform(0.1, 1.0), 3)]), "nll": rng.choice([0.0, round(rng.uniform(0.1, 1.0), 3)])}
    parts = {"f32": [], "bf16": []}
    for _ in range(rng.randint(1, 4)):
        n = _log(rng, 1, 1 << 25)
        parts[rng.choice(["f32", "bf16"])].append("%dx%d" % (n, min(rng.randint(1, 24), max(1, (1 << 26) // n))))
    return {"op": "gradnorm", "f32": ",".join(parts["f32"]), "bf16": ",".join(parts["bf16"]), "packed": rng.random() < 0.5, "norm": rng.choice(["l2", "l2", "max"]), "clip": rng.random() < 0.5}


def _sizes(text):
    return [int(n) for part in text.split(",") if part for n, k in [part.split("x")] for _ in range(int(k))]


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    uniform = lambda *shape: torch.rand(*shape, generator=g, device="cuda")  # noqa: E731
    return {"logprobs": _prepare_logprobs, "clip": _prepare_clip, "pref": _prepare_pref, "gradnorm": _prepare_gradnorm}[case["op"]](case, normal, uniform, g)


def _prepare_logprobs(case, normal, uniform, g):
    n, d, v, t = case["tokens"], case["hidden"], case["vocab"], TYPES[case["type"]]
    s = dict(case)
    w = 0.02 * normal(v, d)
    s["y"] = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    h = normal(n, d)
    h = h / h.square().mean(1, keepdim=True).sqrt()
    # a trained model's targets: from as likely as any other token to nearly certain
    at = w[s["y"].long()]
    h = h + 25 * uniform(n, 1) * at / at.norm(dim=1, keepdim=True)
    s["H"], s["W"] = h.to(t).requires_grad_(own), w.to(t).requires_grad_(own)
    s["g"] = normal(n) / n * (uniform(n) < case["live"])
    return s


def _mask(batch, length, uniform):
    """Behind a prompt and in front of the padding; one sequence in sixteen or so has no token at all."""
    start = (uniform(batch, 1) * 0.25 * length).floor()
    end = start + ((0.3 + 0.7 * uniform(batch, 1)) * (length - start)).ceil() * (uniform(batch, 1) > 1 / 16)
    j = torch.arange(length, device="cuda")
    return ((j >= start) & (j < end)).view(-1)


def _logs(n, normal, uniform, keep):
    """Log-probabilities of the policy: many tokens all but certain, some unlikely; padding's targets have none."""
    lp = -(4 * uniform(n) ** 4 + normal(n).abs() * 0.2)
    return torch.where(keep | (uniform(n) < 0.5), lp, math.nan)


def _prepare_clip(case, normal, uniform, g):
    b, n = case["sequences"], case["sequences"] * case["length"]
    s = dict(case)
    keep = _mask(b, case["length"], uniform)
    s["mask"] = keep.to(torch.uint8)
    s["lp"] = _logs(n, normal, uniform, keep)
    # the policy has moved by some steps since the rollout, and further from the reference
    s["old"] = s["lp"] + 0.15 * normal(n)
    s["ref"] = s["lp"] + 0.3 * normal(n) if case["beta"] else None
    s["advantages"] = normal(b if case["adv"] == "sequence" else n)
    return s


def _prepare_pref(case, normal, uniform, g):
    n = 2 * case["pairs"] * case["length"]
    s = dict(case)
    keep = _mask(2 * case["pairs"], case["length"], uniform)
    s["mask"] = keep.to(torch.uint8)
    s["lp"] = _logs(n, normal, uniform, keep)
    s["ref"] = s["lp"] + 0.1 * normal(n) if case["reference"] else None
    return s


def _prepare_gradnorm(case, normal, uniform, g):
    s = dict(case)
    views = []
    for kind in ("f32", "bf16"):
        at, places = 0, []
        for n in _sizes(case[kind]):
            places.append((at, n))
            at += n if case["packed"] else -(-n // 128) * 128
        flat = torch.zeros(at + 1, device="cuda", dtype=TYPES[kind])  # nothing between the tensors, and behind the last
        for o, n in places:
            flat[o:o + n] = (1e-3 * normal(n)).to(TYPES[kind])
            views.append(flat[o:o + n])
        s["flat_" + kind] = flat
    if own:
        import grpo_policy_loss_amd as gp

        s["plan"] = gp.grad_plan(views)  # what a training loop makes once, for the gradients that it keeps
    return s


# ---------------------------------------------------------------- one pass


def run(state):
    if own:
        return {"logprobs": _own_logprobs, "clip": _own_clip, "pref": _own_pref, "gradnorm": _own_gradnorm}[state["op"]](state)
    return {"logprobs": _plain_logprobs, "clip": _plain_clip, "pref": _plain_pref, "gradnorm": _plain_gradnorm}[state["op"]](state)


def _own_logprobs(s):
    import grpo_policy_loss_amd as gp

    lp = gp.grpo_logprobs(s["H"], s["W"], s["y"], chunk=8192, opts={"temperature": s["temperature"]})
    dh, dw = torch.autograd.grad(lp, (s["H"], s["W"]), s["g"])
    return {"lp": lp.detach(), "dh": dh, "dw": dw}


def _own_clip(s):
    import grpo_policy_loss_amd as gp

    how = {"old_lp": s["old"], "ref_lp": s["ref"], "beta": s["beta"], "clip_low": s["low"], "clip_high": s["high"], "clip_dual": s["dual"],
           "ratio": gp.RATIO_TOKEN if s["level"] == "token" else gp.RATIO_SEQUENCE, "kl_estimator": gp.KL_REVERSE if s["kl"] == "reverse" else gp.KL_FORWARD,
           "aggregation": gp.AGG_TOKEN_MEAN if s["mean"] == "token" else gp.AGG_SEQUENCE_MEAN}
    loss, stats, weights = gp.grpo_clip_loss_fwd(s["lp"], s["mask"], s["advantages"], s["sequences"], s["length"], **how)
    return {"loss": loss, "stats": stats, "grad": gp.grpo_clip_loss_bwd(s["lp"], s["mask"], s["advantages"], weights, s["sequences"], s["length"], **how)}


def _own_pref(s):
    import grpo_policy_loss_amd as gp

    kind = {"sigmoid": gp.PREF_SIGMOID, "hinge": gp.PREF_HINGE, "square": gp.PREF_SQUARE}[s["kind"]]
    loss, rewards, weights = gp.grpo_pref_loss_fwd(s["lp"], s["mask"], s["pairs"], s["length"], ref_lp=s["ref"], beta=PREF_BETA, kind=kind, length_mean=s["averaged"],
                                                   label_smoothing=s["smoothing"], margin=s["margin"], nll_weight=s["nll"])
    return {"loss": loss, "rewards": rewards, "grad": gp.grpo_pref_loss_bwd(s["mask"], weights, s["pairs"], s["length"])}


def _own_gradnorm(s):
    import grpo_policy_loss_amd as gp

    norm, scale = gp.grpo_grad_norm(s["plan"], max_norm=MAX_NORM, kind=gp.GRAD_NORM_L2 if s["norm"] == "l2" else gp.GRAD_NORM_MAX)
    out = {"norm": norm, "scale": scale}
    if s["clip"]:
        gp.grpo_grad_clip(s["plan"], scale)
        out |= {"f32": s["flat_f32"], "bf16": s["flat_bf16"]}
    return out


def _plain_logprobs(s):
    with torch.no_grad():
        h, w, y, k = s["H"].float(), s["W"].float(), s["y"].long()[:, None], 1 / s["temperature"]
        z = h @ w.t() * k
        lp = z - z.amax(1, keepdim=True)
        lp = lp - lp.exp().sum(1, keepdim=True).log()
        # g (onehot - p), a row without a gradient left out of what it may hold
        dz = lp.exp().scatter_add(1, y, torch.full_like(s["g"][:, None], -1.0)) * -s["g"][:, None]
        dz = torch.where(s["g"][:, None] == 0, 0.0, dz) * k
        return {"lp": lp.gather(1, y)[:, 0], "dh": (dz @ w).to(s["H"].dtype), "dw": (dz.t() @ h).to(s["W"].dtype)}


def _plain_clip(s):
    b, n = s["sequences"], s["length"]
    keep = s["mask"].view(b, n) != 0
    # in 64 bits: which side of the clip's border a ratio is on, and long sums
    wide = lambda x: torch.where(keep, x.view(b, n).double(), 0.0)  # noqa: E731
    lp = wide(s["lp"])
    d = lp - wide(s["old"])
    count = keep.sum(1, keepdim=True)
    adv = s["advantages"].double().view(b, 1) if s["adv"] == "sequence" else wide(s["advantages"])
    ratio = d.exp() if s["level"] == "token" else (d.sum(1, keepdim=True) / count.clamp(min=1)).exp()
    above = (adv >= 0) & (ratio > 1 + s["high"])
    below = (adv < 0) & (ratio < 1 - s["low"])
    far = (adv < 0) & (ratio > (s["dual"] or math.inf))
    used = torch.where(above, 1 + s["high"], torch.where(below, 1 - s["low"], torch.where(far, s["dual"], ratio)))
    loss = -adv * used
    slope = torch.where(above | below | far, 0.0, -adv * ratio)
    kl = torch.zeros_like(d)
    if s["beta"]:
        x = wide(s["ref"]) - lp
        kl = x.expm1() - x if s["kl"] == "reverse" else x.exp() * x - x.expm1()
        loss = loss + s["beta"] * kl
        slope = slope + s["beta"] * (-x.expm1() if s["kl"] == "reverse" else -x * x.exp())
    total = keep.sum().clamp(min=1)
    weight = keep / total if s["mean"] == "token" else keep / (b * count.clamp(min=1))
    mean = lambda x: (x * keep).sum() / total  # noqa: E731
    stats = torch.stack([mean(kl), mean(below.double()), mean((above | far).double()), mean(ratio - 1 - ratio.log())])
    return {"loss": (weight * loss).sum().view(1).float(), "stats": stats.float(), "grad": (weight * slope).float().view(-1)}


def _plain_pref(s):
    p, n = s["pairs"], s["length"]
    keep = s["mask"].view(2 * p, n) != 0
    count = keep.sum(1).clamp(min=1)
    lp = torch.where(keep, s["lp"].view(2 * p, n), 0.0)
    r = lp if s["ref"] is None else lp - torch.where(keep, s["ref"].view(2 * p, n), 0.0)
    total = r.sum(1, dtype=torch.float64)  # thousands of tokens
    if s["averaged"]:
        total = total / count
    h = (total.view(p, 2) * torch.tensor([1.0, -1.0], dtype=torch.float64, device="cuda")).sum(1)
    x = PREF_BETA * h - s["margin"]
    softplus = lambda x: x.clamp(min=0) + (-x.abs()).exp().log1p()  # noqa: E731
    if s["kind"] == "sigmoid":
        loss = (1 - s["smoothing"]) * softplus(-x) + s["smoothing"] * softplus(x)
        slope = PREF_BETA * (1 / (1 + (-x).exp()) - (1 - s["smoothing"]))
    elif s["kind"] == "hinge":
        loss = (1 - x).clamp(min=0)
        slope = torch.where(x < 1, -PREF_BETA, 0.0).double()
    else:
        off = h - s["margin"] - 1 / (2 * PREF_BETA)
        loss, slope = off * off, 2 * off
    each = torch.stack([slope, -slope], 1).view(-1) / p
    if s["averaged"]:
        each = each / count
    if s["nll"]:
        chosen = (torch.arange(2 * p, device="cuda") % 2 == 0) * s["nll"] / count
        loss = loss - (lp.sum(1, dtype=torch.float64) * chosen).view(p, 2)[:, 0]
        each = each - chosen / p
    return {"loss": loss.mean().view(1).float(), "rewards": (PREF_BETA * total).float(), "grad": (keep * each.float()[:, None]).view(-1)}


def _plain_gradnorm(s):
    # all tensors at once
    a, b = s["flat_f32"], s["flat_bf16"].float()
    if s["norm"] == "l2":
        norm = (a.square().sum(dtype=torch.float64) + b.square().sum(dtype=torch.float64)).sqrt()
    else:
        norm = torch.maximum(a.abs().max(), b.abs().max()).double()
    scale = (MAX_NORM / (norm + 1e-6)).clamp(max=1).float().view(1)
    out = {"norm": norm.float().view(1), "scale": scale}
    if s["clip"]:
        a.mul_(scale)
        s["flat_bf16"].copy_(b * scale)
        out |= {"f32": a, "bf16": s["flat_bf16"]}
    return out


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "logprobs":
        n, d, v, b = case["tokens"], case["hidden"], case["vocab"], 4 if case["type"] == "f32" else 2
        # H, W, targets and gradients in; log-probabilities and both gradients out; one product forward, and of live tokens three backward
        return {"bytes": 2 * (n + v) * d * b + 12 * n, "flops": int(2 * n * v * d * (1 + 3 * case["live"]))}
    if case["op"] == "clip":
        n, per = case["sequences"] * case["length"], case["sequences"] if case["adv"] == "sequence" else case["sequences"] * case["length"]
        return {"bytes": n * (4 + 4 + (4 if case["beta"] else 0) + 1 + 4) + 4 * per, "flops": 60 * n}
    if case["op"] == "pref":
        n = 2 * case["pairs"] * case["length"]
        return {"bytes": n * (4 + (4 if case["reference"] else 0) + 1 + 4) + 8 * case["pairs"], "flops": 4 * n}
    n = sum(_sizes(case["f32"])) * 4 + sum(_sizes(case["bf16"])) * 2
    return {"bytes": n * (2 if case["clip"] else 1), "flops": 2 * (sum(_sizes(case["f32"])) + sum(_sizes(case["bf16"])))}


# ---------------------------------------------------------------- from the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "clip": _exact_clip, "pref": _exact_pref, "gradnorm": _exact_gradnorm}[case["op"]](s)


def _exact_logprobs(s):
    """The gradient of sum g lp with respect to the logits, then through the product."""
    h, w = s["H"].detach().double(), s["W"].detach().double()
    z = torch.mm(h, w.t()).div_(s["temperature"])
    rows, y = torch.arange(z.shape[0], device="cuda"), s["y"].long()
    lp = z[rows, y] - torch.logsumexp(z, 1)
    g = s["g"].double()
    dz = torch.softmax(z, 1).mul_(-g[:, None])
    dz[rows, y] += g
    dz /= s["temperature"]
    return {"lp": lp, "dh": torch.mm(dz, w), "dw": torch.mm(dz.t(), h)}


def _exact_clip(s):
    """The objective as minima of products, sequence by sequence over their own tokens; its gradient by differentiation."""
    b, n = s["sequences"], s["length"]
    keep = s["mask"].bool()
    of = torch.arange(b, device="cuda").repeat_interleave(n)[keep]
    lp = s["lp"].double()[keep].requires_grad_()
    adv = s["advantages"].double()[of] if s["adv"] == "sequence" else s["advantages"].double()[keep]
    count = torch.zeros(b, dtype=torch.float64, device="cuda").index_add(0, of, torch.ones_like(lp.detach())).clamp(min=1)
    d = lp - s["old"].double()[keep]
    if s["level"] == "sequence":
        d = (torch.zeros(b, dtype=torch.float64, device="cuda").index_add(0, of, d) / count)[of]
    ratio = d.exp()
    clipped = ratio.clamp(1 - s["low"], 1 + s["high"])
    objective = torch.minimum(ratio * adv, clipped * adv)
    bounded = torch.maximum(objective, s["dual"] * adv) if s["dual"] else objective
    objective = torch.where(adv < 0, bounded, objective)
    kl = torch.zeros_like(d)
    if s["beta"]:
        x = s["ref"].double()[keep] - lp
        kl = x.exp() - x - 1 if s["kl"] == "reverse" else x.exp() * x - (x.exp() - 1)
    share = (1 / count / b)[of] if s["mean"] == "sequence" else torch.full_like(d, 1 / max(1, lp.numel()))
    loss = ((s["beta"] * kl - objective) * share).sum()
    grad = torch.zeros(b * n, dtype=torch.float64, device="cuda")
    if lp.numel():
        grad[keep] = torch.autograd.grad(loss, lp)[0]
    with torch.no_grad():
        below = (adv < 0) & (ratio < 1 - s["low"])
        above = ((adv >= 0) & (ratio > 1 + s["high"])) | ((adv < 0) & (ratio > s["dual"]) if s["dual"] else torch.zeros_like(below))
        stats = [v.double().sum() / max(1, lp.numel()) for v in (kl, below, above, ratio - 1 - d)]
    return {"loss": loss.detach().view(1), "stats": torch.stack(stats), "grad": grad}


def _exact_pref(s):
    p, n = s["pairs"], s["length"]
    keep = s["mask"].bool()
    of = torch.arange(2 * p, device="cuda").repeat_interleave(n)[keep]
    lp = s["lp"].double()[keep].requires_grad_()
    per = lambda x: torch.zeros(2 * p, dtype=torch.float64, device="cuda").index_add(0, of, x)  # noqa: E731
    count = per(torch.ones_like(lp.detach())).clamp(min=1)
    total = per(lp if s["ref"] is None else lp - s["ref"].double()[keep])
    total = total / count if s["averaged"] else total
    h = total[0::2] - total[1::2]
    x = PREF_BETA * h - s["margin"]
    if s["kind"] == "sigmoid":
        loss = torch.logaddexp(torch.zeros_like(x), -x) * (1 - s["smoothing"]) + torch.logaddexp(torch.zeros_like(x), x) * s["smoothing"]
    elif s["kind"] == "hinge":
        loss = torch.relu(1 - x)
    else:
        loss = (h - s["margin"] - 0.5 / PREF_BETA) ** 2
    loss = (loss - s["nll"] * (per(lp) / count)[0::2]).sum() / p
    grad = torch.zeros(2 * p * n, dtype=torch.float64, device="cuda")
    if lp.numel():
        grad[keep] = torch.autograd.grad(loss, lp)[0]
    return {"loss": loss.detach().view(1), "rewards": PREF_BETA * total.detach(), "grad": grad}


def _exact_gradnorm(s):
    flats = [s["flat_f32"].double(), s["flat_bf16"].double()]
    if s["norm"] == "l2":
        norm = torch.cat([x.view(1, -1) @ x.view(-1, 1) for x in flats]).sum().sqrt()
    else:
        norm = torch.cat(flats).abs().amax()
    scale = torch.where(norm + 1e-6 > MAX_NORM, MAX_NORM / (norm + 1e-6), torch.ones_like(norm))
    out = {"norm": norm.view(1), "scale": scale.view(1)}
    if s["clip"]:
        out |= {"f32": flats[0] * scale, "bf16": flats[1] * scale}
    return out
