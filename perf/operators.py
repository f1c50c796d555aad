"""The operators around the policy loss as they are called in a training step and a rollout: the final norm
(forward and backward), the optimizer's step and the sampling of the next token.

`run` computes each in its plain form, or with `own` through grpo_policy_loss_amd. Cases are plain dicts:

  op "norm":   kind "rms" or "layer", pass "fwd" or "bwd", type, rows, cols, bias
  op "adamw":  sizes "elements x count, ...", type of the parameters, grads, master (float32 copy), bits of the
               moments, packed (tensors at odd offsets of one buffer, or each on a 128-element boundary), clip
  op "sample": type, batch, vocab, temperature, top_k, top_p, min_p; rows (parameters drawn for each row),
               masked (share of the vocabulary at -inf)
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
LR, BETAS, ADAM_EPS, DECAY = 1e-5, (0.9, 0.999), 1e-8, 0.01
BLOCK = 256  # elements of one scale of the 8-bit moments


def listed():
    return [
        # the final norm of one token being generated: a launch's latency
        {"name": "norm token", "op": "norm", "kind": "rms", "pass": "fwd", "type": "bf16", "rows": 1, "cols": 4096, "bias": False},
        # the final norm in front of the loss: 32 completions of 1024 tokens
        {"name": "norm batch", "op": "norm", "kind": "rms", "pass": "fwd", "type": "bf16", "rows": 32768, "cols": 1536, "bias": False},
        # its backward pass at the widest hidden size, with mean and bias
        {"name": "norm batch bwd", "op": "norm", "kind": "layer", "pass": "bwd", "type": "bf16", "rows": 32768, "cols": 4096, "bias": True},
        # float32 with no size a power of two or a multiple of four: rows start at any alignment
        {"name": "norm ragged bwd", "op": "norm", "kind": "layer", "pass": "bwd", "type": "f32", "rows": 4099, "cols": 1537, "bias": True},
        # the head alone: bfloat16 weights with float32 masters and the loss's float32 gradient, clipped
        {"name": "adamw head", "op": "adamw", "sizes": "233373696x1", "type": "bf16", "grads": "f32", "master": True, "bits": 32, "packed": False, "clip": True},
        # the matrices of a layer with moments in 8 bits
        {"name": "adamw 8 bits", "op": "adamw", "sizes": "16777216x4,4096x2", "type": "bf16", "grads": "bf16", "master": False, "bits": 8, "packed": False, "clip": False},
        # many small tensors that lie packed in one buffer
        {"name": "adamw many", "op": "adamw", "sizes": "1536x96,257x32,4099x16,1x8,100003x8", "type": "f32", "grads": "f32", "master": False, "bits": 32, "packed": True, "clip": False},
        # two norm weights: a launch's latency
        {"name": "adamw vectors", "op": "adamw", "sizes": "1536x2", "type": "bf16", "grads": "f32", "master": False, "bits": 32, "packed": False, "clip": False},
        # one token from the whole distribution
        {"name": "sample one", "op": "sample", "type": "f32", "batch": 1, "vocab": 151936, "temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, "rows": False, "masked": 0.0},
        # a step of a training rollout: the policy's own distribution
        {"name": "sample rollout", "op": "sample", "type": "f32", "batch": 256, "vocab": 128256, "temperature": 0.9, "top_k": 0, "top_p": 1.0, "min_p": 0.0, "rows": False, "masked": 0.0},
        # a step of an evaluation: bfloat16 logits, so many of them equal
        {"name": "sample top-k top-p", "op": "sample", "type": "bf16", "batch": 32, "vocab": 151936, "temperature": 0.7, "top_k": 50, "top_p": 0.95, "min_p": 0.0, "rows": False, "masked": 0.01},
        # requests with parameters of their own
        {"name": "sample requests", "op": "sample", "type": "f32", "batch": 64, "vocab": 201088, "temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, "rows": True, "masked": 0.01},
    ]


def _log(rng, low, high):
    """A whole number, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "adamw", "sample"])
    if op == "norm":
        cols = _log(rng, 16, 16384)
        if rng.random() < 0.5:
            cols = cols // 8 * 8
        rows = _log(rng, 1, max(1, min(65536, 32768 * 4096 // cols)))
        kind = rng.choice(["rms", "layer"])
        return {"op": "norm", "kind": kind, "pass": rng.choice(["fwd", "bwd"]), "type": rng.choice(["f32", "bf16"]) if rows * cols < 1 << 26 else "bf16",
                "rows": rows, "cols": cols, "bias": kind == "layer" and rng.random() < 0.7}
    if op == "adamw":
        bits = rng.choice([32, 8])
        sizes = []
        for _ in range(rng.randint(1, 3)):
            n = _log(rng, 1, 1 << 24)
            sizes.append("%dx%d" % (n, min(rng.randint(1, 8), max(1, (1 << 25) // n))))
        kind = rng.choice(["f32", "bf16"])
        return {"op": "adamw", "sizes": ",".join(sizes), "type": kind, "grads": rng.choice(["f32", "bf16"]) if kind == "bf16" else "f32",
                "master": kind == "bf16" and rng.random() < 0.5, "bits": bits, "packed": rng.random() < 0.5, "clip": rng.random() < 0.5}
    batch = _log(rng, 1, 256)
    return {"op": "sample", "type": rng.choice(["f32", "bf16"]), "batch": batch, "vocab": _log(rng, 2, 201088 if batch <= 160 else 128256),
            "temperature": round(rng.uniform(0.3, 1.5), 3), "top_k": rng.choice([0, 1, _log(rng, 1, 2000)]), "top_p": rng.choice([1.0, round(rng.uniform(0.3, 0.99), 3)]),
            "min_p": rng.choice([0.0, round(rng.uniform(0.001, 0.2), 4)]), "rows": rng.random() < 0.3, "masked": rng.choice([0.0, 0.01, 0.3])}


def _sizes(case):
    return [int(n) for part in case["sizes"].split(",") for n, k in [part.split("x")] for _ in range(int(k))]


def _offsets(case):
    """Each tensor's place in the buffers, and the buffers' length."""
    at, offsets = 0, []
    for n in _sizes(case):
        offsets.append(at)
        at += n if case["packed"] else -(-n // 128) * 128
    return offsets, at


def _scale_offsets(case):
    at, offsets = 0, []
    for n in _sizes(case):
        offsets.append(at)
        at += -(-n // BLOCK)
    return offsets, at


def _views(flat, offsets, sizes):
    return [flat[o:o + n] for o, n in zip(offsets, sizes)]


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    return {"norm": _prepare_norm, "adamw": _prepare_adamw, "sample": _prepare_sample}[case["op"]](case, normal, g)


def _prepare_norm(case, normal, g):
    rows, cols, t = case["rows"], case["cols"], TYPES[case["type"]]
    s = dict(case)
    # a residual stream: a size that differs from row to row, and an offset
    s["x"] = (normal(rows, cols) * (0.5 + 2 * torch.rand(rows, 1, generator=g, device="cuda")) + 0.1 * normal(rows, 1)).to(t)
    s["weight"] = (1 + 0.1 * normal(cols)).to(t)
    s["b"] = (0.1 * normal(cols)).to(t) if case["bias"] else None
    if case["pass"] == "bwd":
        s["dy"] = (normal(rows, cols) * 1e-2).to(t)
        s["mean"], s["rstd"] = _statistics(s["x"].double(), case["kind"])
    return s


def _statistics(x, kind):
    mean = x.mean(1) if kind == "layer" else None
    rstd = ((x if mean is None else x - mean[:, None]).square().mean(1) + EPS).rsqrt()
    return None if mean is None else mean.float(), rstd.float()


def _prepare_adamw(case, normal, g):
    s = dict(case)
    sizes, (offsets, n) = _sizes(case), _offsets(case)
    weights = 0.02 * normal(n)
    inside = torch.zeros(n, device="cuda")  # nothing between the tensors
    for o, k in zip(offsets, sizes):
        inside[o:o + k] = 1
    weights *= inside
    s["flat"] = {"p": weights.to(TYPES[case["type"]]), "g": (1e-3 * normal(n) * inside).to(TYPES[case["grads"]])}
    if case["master"]:
        s["flat"]["master"] = s["flat"]["p"].float() + 1e-5 * normal(n) * inside
    m, v = 3e-4 * normal(n) * inside, 1e-6 * normal(n).square() * inside
    if case["bits"] == 32:
        s["flat"]["m"], s["flat"]["v"] = m, v
    else:
        scales, blocks = _scale_offsets(case)
        s["flat"]["m_codes"] = torch.zeros(n, dtype=torch.int8, device="cuda")
        s["flat"]["v_codes"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        s["flat"]["m_scales"], s["flat"]["v_scales"] = (torch.zeros(blocks, device="cuda") for _ in range(2))
        for o, k, b in zip(offsets, sizes, scales):
            for name, x in (("m", m), ("v", v)):
                c, a = _encode(x[o:o + k].double(), name == "v")
                s["flat"][name + "_codes"][o:o + k] = c
                s["flat"][name + "_scales"][b:b + a.numel()] = a
        for name in ("m_scales", "v_scales"):
            s[name] = _views(s["flat"][name], scales, [-(-k // BLOCK) for k in sizes])
    for name, flat in s["flat"].items():
        if not name.endswith("scales"):
            s["masters" if name == "master" else name] = _views(flat, offsets, sizes)
    s["clip_by"] = torch.full((1,), 0.37, device="cuda") if case["clip"] else None
    s["step"] = 100
    if own:
        import grpo_policy_loss_amd as gp

        if case["bits"] == 8:
            s["moments"] = {k: [gp.Moment8(c, a) for c, a in zip(s[k + "_codes"], s[k + "_scales"])] for k in "mv"}
        else:
            s["moments"] = {k: s[k] for k in "mv"}
        # what a training loop makes once, for the tensors that it keeps
        s["plan"] = gp.adamw_plan(s["p"], s["g"], s["moments"]["m"], s["moments"]["v"], master=s.get("masters"))
    return s


def _prepare_sample(case, normal, g):
    s = dict(case)
    batch, vocab = case["batch"], case["vocab"]
    uniform = lambda *shape: torch.rand(*shape, generator=g, device="cuda")  # noqa: E731
    logits = 2.5 * normal(batch, vocab)
    # a language model's logits: a few tokens stand out, by more in some rows than in others
    few = max(1, min(12, vocab // 4))
    at = torch.randint(0, vocab, (batch, few), generator=g, device="cuda")
    logits.scatter_add_(1, at, uniform(batch, few) * 14 * uniform(batch, 1))
    if case["masked"]:
        off = uniform(batch, vocab) < case["masked"]
        off[:, 0] = False
        logits.masked_fill_(off, float("-inf"))
    s["logits"] = logits.to(TYPES[case["type"]])
    s["u"] = uniform(batch)
    if case["rows"]:
        pick = uniform(4, batch)
        s["temperature"] = 0.3 + 1.2 * uniform(batch)
        s["top_k"] = torch.where(pick[0] < 0.5, torch.zeros_like(pick[0]), 1 + 200 * uniform(batch)).to(torch.int32)
        s["top_p"] = torch.where(pick[1] < 0.4, torch.ones_like(pick[1]), 0.5 + 0.49 * uniform(batch))
        s["min_p"] = torch.where(pick[2] < 0.6, torch.zeros_like(pick[2]), 0.2 * uniform(batch))
    return s


# ---------------------------------------------------------------- one pass


def run(state):
    if own:
        return {"norm": _own_norm, "adamw": _own_adamw, "sample": _own_sample}[state["op"]](state)
    return {"norm": _plain_norm, "adamw": _plain_adamw, "sample": _plain_sample}[state["op"]](state)


def _own_norm(s):
    import grpo_policy_loss_amd as gp

    kind = gp.NORM_RMS if s["kind"] == "rms" else gp.NORM_LAYER
    if s["pass"] == "fwd":
        y, mean, rstd = gp.grpo_norm_fwd(s["x"], s["weight"], s["b"], eps=EPS, kind=kind)
        return {"y": y, "mean": mean, "rstd": rstd}
    dx, dw, db = gp.grpo_norm_bwd(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], kind=kind, bias=s["bias"])
    return {"dx": dx, "dw": dw, "db": db}


def _own_adamw(s):
    import grpo_policy_loss_amd as gp

    s["step"] += 1
    gp.grpo_adamw(s["plan"], step=s["step"], lr=LR, betas=BETAS, eps=ADAM_EPS, weight_decay=DECAY, grad_scale=s["clip_by"])
    out = {k: s["flat"][k] for k in ("p", "master") if k in s["flat"]}
    if s["bits"] == 32:
        return out | {"m": s["flat"]["m"], "v": s["flat"]["v"]}
    return out | {k: [gp.dequantize_moment(x) for x in s["moments"][k]] for k in "mv"}


def _own_sample(s):
    import grpo_policy_loss_amd as gp

    token, lp = gp.grpo_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    return {"token": token, "lp": lp}


def _plain_norm(s):
    x, w, t = s["x"].float(), s["weight"].float(), s["x"].dtype
    if s["pass"] == "fwd":
        mean = x.mean(1) if s["kind"] == "layer" else None
        d = x if mean is None else x - mean[:, None]
        rstd = (d.square().mean(1) + EPS).rsqrt()
        y = d * rstd[:, None] * w
        return {"y": (y if s["b"] is None else y + s["b"].float()).to(t), "mean": mean, "rstd": rstd}
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (x if s["mean"] is None else x - s["mean"][:, None]) * rstd
    gw = dy * w
    dx = gw - xh * (gw * xh).mean(1, keepdim=True)
    if s["kind"] == "layer":
        dx = dx - gw.mean(1, keepdim=True)
    return {"dx": (dx * rstd).to(t), "dw": (dy * xh).sum(0), "db": dy.sum(0) if s["bias"] else None}


def _encode(x, positive):
    """Codes and scales of a moment in 8 bits, from values in 64."""
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    scale = b.abs().amax(1).float()
    share = torch.where(scale[:, None] > 0, b.abs() / scale.double()[:, None], torch.zeros_like(b))
    if positive:
        c = torch.where(b > 0, (255 * share.sqrt().sqrt() + 0.5).floor().clamp(1, 255), torch.zeros_like(b)).to(torch.uint8)
    else:
        c = (b.sign() * (127 * share.sqrt() + 0.5).floor().clamp(max=127)).to(torch.int8)
    return c.view(-1)[:n], scale


def _decode(codes, scales):
    c = codes.double()
    c = (c / 255) ** 4 if codes.dtype == torch.uint8 else c.sign() * (c / 127).square()
    return c * scales.double().repeat_interleave(BLOCK)[:codes.numel()]


def _update(w, g, m, v, t, clip_by):
    """The moments and weights after step t, in the type of g, m and v."""
    b1, b2 = BETAS
    if clip_by is not None:
        g = g * clip_by
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    return w * (1 - LR * DECAY) - (LR / (1 - b1 ** t)) * m / ((v / (1 - b2 ** t)).sqrt() + ADAM_EPS), m, v


def _plain_adamw(s):
    s["step"] += 1
    flat = s["flat"]
    main = "master" if s["master"] else "p"
    out = {k: flat[k] for k in ("p", "master") if k in flat}
    if s["bits"] == 32:  # all tensors at once
        for to, x in zip((main, "m", "v"), _update(flat[main].float(), flat["g"].float(), flat["m"], flat["v"], s["step"], s["clip_by"])):
            flat[to].copy_(x)
        if s["master"]:
            flat["p"].copy_(flat["master"])
        return out | {"m": flat["m"], "v": flat["v"]}
    values = {"m": [], "v": []}
    clip_by = None if s["clip_by"] is None else s["clip_by"].double()
    for i, w in enumerate(s["masters" if s["master"] else "p"]):
        # in 64 bits: a code goes by which side of a border its value is on
        m, v = (_decode(s[k + "_codes"][i], s[k + "_scales"][i]) for k in "mv")
        new, m, v = _update(w.double(), s["g"][i].double(), m, v, s["step"], clip_by)
        w.copy_(new)
        if s["master"]:
            s["p"][i].copy_(w)
        for k, x in (("m", m), ("v", v)):
            c, a = _encode(x, k == "v")
            s[k + "_codes"][i].copy_(c)
            s[k + "_scales"][i].copy_(a)
            values[k].append(_decode(c, a).float())
    return out | values


def _plain_sample(s):
    x = s["logits"].double()  # in 64 bits: a token goes by which side of a border u is on
    batch, vocab = x.shape
    per_row = lambda v: v.double()[:, None] if torch.is_tensor(v) else float(v)  # noqa: E731
    T, k, p, least = (per_row(s[n]) for n in ("temperature", "top_k", "top_p", "min_p"))
    z = x / T
    w = (z - z.amax(1, keepdim=True)).exp()
    mass = w
    if s["rows"] or s["top_k"] or s["top_p"] < 1 or s["min_p"]:
        order = x.sort(dim=1, descending=True, stable=True).indices  # equal ones by index
        ws = w.gather(1, order)
        off = lambda v, none: (v == none) if torch.is_tensor(v) else torch.tensor(v == none, device=x.device)  # noqa: E731
        keep = ((torch.arange(vocab, device=x.device) < k) | off(k, 0)).expand(batch, vocab)
        ws = ws * keep
        before = ws.cumsum(1) - ws
        keep = keep & ((before < p * ws.sum(1, keepdim=True)) | off(p, 1)) & (ws >= least)
        mass = w * torch.zeros_like(keep).scatter_(1, order, keep)
    run_up = mass.cumsum(1)
    target = s["u"].double()[:, None] * run_up[:, -1:]
    token = (run_up <= target).sum(1, keepdim=True).clamp(max=vocab - 1)
    lp = z.gather(1, token) - z.logsumexp(1, keepdim=True)
    return {"token": token[:, 0].to(torch.int32), "lp": lp[:, 0].float()}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "norm":
        n, b, c = case["rows"] * case["cols"], 4 if case["type"] == "f32" else 2, case["cols"]
        stats = 4 * case["rows"] * (2 if case["kind"] == "layer" else 1)
        if case["pass"] == "fwd":
            return {"bytes": 2 * n * b + stats + c * b * (2 if case["bias"] else 1), "flops": 8 * n}
        return {"bytes": 3 * n * b + stats + c * (b + 4 * (2 if case["bias"] else 1)), "flops": 14 * n}
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        p, g = (2 if case[k] == "bf16" else 4 for k in ("type", "grads"))
        weights = p + 8 if case["master"] else 2 * p
        # in 8 bits: codes and scales in and out, and the values that they stand for out
        moments = 16 if case["bits"] == 32 else 4 + 16 / BLOCK + 8
        return {"bytes": n * (weights + g + moments), "flops": 16 * n}
    n = case["batch"] * case["vocab"]
    return {"bytes": n * (4 if case["type"] == "f32" else 2) + case["batch"] * (12 + (16 if case["rows"] else 0)), "flops": 5 * n}


# ---------------------------------------------------------------- from the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "adamw": _exact_adamw, "sample": _exact_sample}[case["op"]](s)


def _exact_norm(s):
    """The gradients as those of the formula, by the chain rule through mean and variance."""
    x, w = s["x"].double(), s["weight"].double()
    cols = x.shape[1]
    if s["pass"] == "fwd":
        mean = x.sum(1) / cols if s["kind"] == "layer" else None
        c = x if mean is None else x - mean.unsqueeze(1)
        sigma = ((c * c).sum(1) / cols + EPS).sqrt()
        y = c / sigma.unsqueeze(1) * w
        if s["b"] is not None:
            y = y + s["b"].double()
        return {"y": y, "mean": mean, "rstd": 1 / sigma}
    dy, r = s["dy"].double(), s["rstd"].double().unsqueeze(1)
    c = x if s["mean"] is None else x - s["mean"].double().unsqueeze(1)
    dw = torch.einsum("ij,ij->j", dy, c * r)
    dxh = dy * w
    # y = c r w with r = (mean c^2 + eps)^(-1/2): dr = -r^3 c dc / cols, and dc = dx - mean dx
    dc = dxh * r - c * r ** 3 * ((dxh * c).sum(1, keepdim=True) / cols)
    if s["kind"] == "layer":
        # sum_j c_j = 0 leaves only the first term's mean
        dc = dc - (dxh * r).sum(1, keepdim=True) / cols
    return {"dx": dc, "dw": dw, "db": dy.sum(0) if s["bias"] else None}


def _exact_adamw(s):
    t = s["step"] + 1
    wide = {k: x.double() for k, x in s["flat"].items() if k in ("p", "g", "m", "v", "master")}
    sizes, (offsets, n) = _sizes(s), _offsets(s)
    if s["bits"] == 8:
        wide["m"], wide["v"] = torch.zeros(2, n, dtype=torch.float64, device="cuda")
        for i, (o, k) in enumerate(zip(offsets, sizes)):
            block = torch.arange(k, device="cuda") // BLOCK
            c = s["m_codes"][i].double() / 127
            wide["m"][o:o + k] = c * c.abs() * s["m_scales"][i].double()[block]
            wide["v"][o:o + k] = (s["v_codes"][i].double() / 255).square().square() * s["v_scales"][i].double()[block]
    g = wide["g"] if s["clip_by"] is None else wide["g"] * s["clip_by"].double()
    m = torch.lerp(wide["m"], g, 1 - BETAS[0])
    v = torch.lerp(wide["v"], g * g, 1 - BETAS[1])
    w = wide.get("master", wide["p"])
    step = (m / -math.expm1(t * math.log(BETAS[0]))) / ((v / -math.expm1(t * math.log(BETAS[1]))).sqrt() + ADAM_EPS)
    new = w - LR * (step + DECAY * w)
    out = {"p": new} | ({"master": new.clone()} if s["master"] else {})
    if s["bits"] == 32:
        return out | {"m": m, "v": v}
    values = {"m": [], "v": []}
    for o, k in zip(offsets, sizes):
        for name, x, top, power in (("m", m, 127, 2), ("v", v, 255, 4)):
            x = x[o:o + k]
            block = torch.arange(k, device="cuda") // BLOCK
            scale = torch.zeros(int(block[-1]) + 1, dtype=torch.float64, device="cuda")
            scale = scale.scatter_reduce(0, block, x.abs(), "amax").float().double()[block]
            share = torch.where(scale > 0, x.abs() / scale, 0.0)
            c = torch.floor(top * share.pow(1 / power) + 0.5).clamp(max=top)
            if name == "v":
                c = torch.where(x > 0, c.clamp(min=1), c)
            values[name].append(torch.sign(x) * (c / top).pow(power) * scale)
    return out | values


def _exact_sample(s):
    """Row by row on the host, from the sorted tokens."""
    batch, vocab = s["logits"].shape
    logits, u = s["logits"].double().cpu().numpy(), s["u"].double().cpu().numpy()
    of = lambda name: (s[name].double().cpu().numpy() if torch.is_tensor(s[name]) else np.full(batch, float(s[name])))  # noqa: E731
    T, top_k, top_p, min_p = (of(n) for n in ("temperature", "top_k", "top_p", "min_p"))
    tokens, lps = np.zeros(batch, np.int32), np.zeros(batch)
    for i in range(batch):
        z = logits[i] / T[i]
        e = np.exp(z - z.max())
        keep = np.ones(vocab, bool)
        if top_k[i] > 0 or top_p[i] < 1 or min_p[i] > 0:
            order = np.argsort(-logits[i], kind="stable")
            if top_k[i] > 0:
                order = order[:int(top_k[i])]
            if top_p[i] < 1:
                up = np.cumsum(e[order])
                order = order[np.concatenate(([0.0], up[:-1])) < top_p[i] * up[-1]]
            order = order[e[order] >= min_p[i]]
            keep[:] = False
            keep[order] = True
        up = np.cumsum(e * keep)
        tokens[i] = min(vocab - 1, np.searchsorted(up, u[i] * up[-1], side="right"))
        lps[i] = z[tokens[i]] - z.max() - np.log(e.sum())
    return {"token": torch.from_numpy(tokens), "lp": torch.from_numpy(lps)}
