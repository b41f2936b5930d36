"""The operators in front of the optimizer step, as they are measured: token log-probabilities, the clipped policy
loss and the preference loss with their gradients, and the global gradient norm with clipping.

A case is one call (or the chain of calls that belongs together) at one size.  With `own` false run() computes the
plain form in elementary torch operations; with `own` true it calls the library.  Logits hold batch x seq tokens of
`vocab` scores; a token whose label is negative is left out of the loss (prompt and padding)."""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_WORKSPACE = 64 << 20
_contexts = {}


def _context(device):
    """The process's library context, made at its first use and kept."""
    if device not in _contexts:
        from newton_schulz_amd import Context
        _contexts[device] = Context(device, _WORKSPACE)
    return _contexts[device]


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _tokens(name, op, dtype, batch, seq, vocab, **more):
    case = {"name": name, "op": op, "dtype": dtype, "batch": batch, "seq": seq, "vocab": vocab,
            "shift": False, "pad": 0, "prompt": 0, "ragged": 0, "temperature": 1.0}
    case.update(more)
    return case


def _clip(name, op, dtype, out, layers, hidden, q, kv, ffn, **more):
    case = {"name": name, "op": op, "dtype": dtype, "out": out, "layers": layers, "hidden": hidden, "q": q, "kv": kv,
            "ffn": ffn, "extra": 0, "max_norm": 1.0}
    case.update(more)
    return case


def listed():
    return [
        # a short answer scored by a small test model: a call whose latency is all there is
        _tokens("score short answer", "logps", "f32", 1, 7, 1000),
        # one sampled token for each of eight sequences, full vocabulary: few long rows
        _tokens("score one token", "logps", "bf16", 8, 1, 151936),
        # the reference policy's scores for four sequences: logits shifted against the labels, no gradient
        _tokens("score batch", "logps", "bf16", 4, 511, 151936, shift=True, prompt=64, ragged=37),
        # maximum likelihood on a vocabulary that is no multiple of anything: rows start at odd addresses
        _tokens("fine-tune odd vocabulary", "logps_grad", "bf16", 2, 1023, 50257, prompt=31, ragged=100),
        # the policy loss of a test model
        _tokens("policy test model", "policy", "f32", 2, 9, 512, prompt=2, ragged=3, reduce="token", kl=0.05,
                per_token=False, old=True),
        # a group of eight answers, mean over each answer, answers of different lengths
        _tokens("policy group", "policy", "bf16", 8, 256, 32000, prompt=40, ragged=23, reduce="sequence", kl=0.04,
                per_token=False, old=True),
        # single-precision logits behind a padded vocabulary, sampled at another temperature, advantages per token
        _tokens("policy f32 padded", "policy", "f32", 3, 333, 32003, pad=61, prompt=10, ragged=50, reduce="token", kl=0.0,
                per_token=True, old=True, temperature=0.7),
        # one long answer over the full vocabulary, first update after sampling is done with (old policy known)
        _tokens("policy long answer", "policy", "bf16", 1, 2048, 151936, prompt=128, reduce="token", kl=0.04,
                per_token=True, old=True),
        # three pairs through a test model
        _tokens("preference test model", "preference", "f32", 6, 33, 4099, prompt=5, ragged=4, kind="sigmoid",
                beta=0.1, smoothing=0.1, average=False),
        # two pairs over the full vocabulary
        _tokens("preference pairs", "preference", "bf16", 4, 400, 151936, prompt=50, ragged=41, kind="sigmoid",
                beta=0.1, smoothing=0.0, average=False),
        # the gradients of one decoder layer, accumulated in single precision, clipped into the optimizer's buffer
        _clip("clip one layer", "clip", "f32", "bf16", 1, 2560, 4096, 1024, 9728),
        # twelve layers' flat gradient buffer: the norm, and the momentum pass that takes its coefficient
        _clip("clip into momentum", "clip_momentum", "bf16", "bf16", 12, 2560, 4096, 1024, 9728),
    ]


_MOST = 2048 * 151936 * 2  # bytes of logits of the largest listed case


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["logps", "logps_grad", "policy", "policy", "preference", "preference", "clip", "clip_momentum"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("clip"):
        hidden, q, kv = (_log_int(rng, 48, 2560) for _ in range(3))
        case = _clip("", op, dtype, rng.choice(["bf16", "f32"]), _log_int(rng, 1, 8), hidden, q, kv, _log_int(rng, 64, 9728),
                     extra=rng.randrange(1, 9), max_norm=round(rng.uniform(0.1, 2.0), 3))
    else:
        vocab, seq, batch = _log_int(rng, 500, 151936), _log_int(rng, 1, 1024), rng.randrange(1, 9)
        if op == "preference":
            batch += batch % 2
        while batch * seq * vocab * (2 if dtype == "bf16" else 4) > _MOST // 2:
            seq = max(1, seq // 2)
        case = _tokens("", op, dtype, batch, seq, vocab, shift=rng.random() < 0.3, pad=rng.choice([0, 0, 8, rng.randrange(1, 64)]),
                       prompt=rng.randrange(0, max(1, seq // 3)), ragged=rng.randrange(0, max(1, seq // 2)),
                       temperature=rng.choice([1.0, 1.0, round(rng.uniform(0.5, 1.5), 2)]))
        if op == "policy":
            case.update(reduce=rng.choice(["token", "sequence", "sum"]), kl=rng.choice([0.0, 0.04, 0.1]),
                        per_token=rng.random() < 0.5, old=rng.random() < 0.8)
        if op == "preference":
            kind = rng.choice(["sigmoid", "sigmoid", "ipo"])
            case.update(kind=kind, beta=round(rng.uniform(0.05, 0.5), 3), average=kind == "ipo",
                        smoothing=rng.choice([0.0, 0.1]) if kind == "sigmoid" else 0.0)
    del case["name"]
    return case


def _shapes(case):
    """The tensors whose gradients are clipped: seven matrices and two vectors a layer, and a few odd ones."""
    h, q, kv, f = case["hidden"], case["q"], case["kv"], case["ffn"]
    layer = [(q, h), (kv, h), (kv, h), (h, q), (f, h), (f, h), (h, f), (h,), (h,)]
    return layer * case["layers"] + [(2 * i + 1,) for i in range(case["extra"])]


def _spans(case):
    """For each sequence the range of tokens that count, the same for every seed."""
    room = case["seq"] - case["prompt"]
    return [(case["prompt"], case["seq"] - (b * case["ragged"]) % max(1, room)) for b in range(case["batch"])]


def _elements(case):
    return sum(math.prod(s) for s in _shapes(case))


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("clip"):
        n, eo = _elements(case), 2 if case["out"] == "bf16" else 4
        if case["op"] == "clip":
            return {"bytes": n * (e + eo), "flops": 3 * n}
        return {"bytes": n * (e + 8 + eo), "flops": 8 * n}
    tokens, vocab = case["batch"] * case["seq"], case["vocab"]
    rows = sum(max(0, hi - lo) for lo, hi in _spans(case))
    if case["op"] == "logps":
        return {"bytes": rows * vocab * e + tokens * 12, "flops": 5 * rows * vocab}
    return {"bytes": rows * vocab * e + tokens * vocab * e + tokens * 28, "flops": 9 * rows * vocab}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    device = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=device).manual_seed(seed * 7919 + 13)
    dt = _DTYPES[case["dtype"]]
    if case["op"].startswith("clip"):
        return _prepare_clip(case, g, device, dt)
    batch, seq, vocab = case["batch"], case["seq"], case["vocab"]
    logits = torch.empty(batch, seq + int(case["shift"]), vocab + case["pad"], dtype=dt, device=device)
    logits.normal_(0.0, 2.0, generator=g)
    logits = logits[:, :seq, :vocab]
    labels = torch.randint(vocab, (batch, seq), generator=g, device=device)
    # a trained policy gives its own tokens more than their share
    lift = torch.rand(batch, seq, 1, generator=g, device=device) * 16.0
    at = labels.unsqueeze(-1)
    logits.scatter_(-1, at, (logits.gather(-1, at).float() + lift).to(dt))
    place = torch.arange(seq, device=device)
    low, high = (torch.tensor(v, device=device).unsqueeze(1) for v in zip(*_spans(case)))
    valid = (place >= low) & (place < high)
    labels.masked_fill_(~valid, -100)
    state = {"case": case, "device": device, "logits": logits, "labels": labels,
             "logps": torch.empty(batch, seq, device=device)}
    if case["op"] == "logps":
        return state
    state["grad"] = torch.empty(batch, seq, vocab, dtype=dt, device=device)

    def noise(scale):
        return torch.randn(batch, seq, generator=g, device=device) * scale

    if case["op"] == "logps_grad":
        # the gradient of the mean negative log-likelihood
        state["grad_logps"] = torch.where(valid, -1.0 / max(1, sum(max(0, hi - lo) for lo, hi in _spans(case))), 0.0).float()
        state["stats"] = torch.empty(batch, seq, 2, device=device)
        return state
    lp = torch.stack([_near_logps(x, y, case["temperature"]) for x, y in zip(logits, labels)])
    if case["op"] == "policy":
        state["advantages"] = noise(1.0) if case["per_token"] else noise(1.0)[:, 0].contiguous()
        state["old"] = torch.where(valid, lp + noise(0.15), 0.0) if case["old"] else None
        state["ref"] = torch.where(valid, lp + noise(0.3), 0.0) if case["kl"] else None
        state["out"] = torch.empty(4, device=device)
    else:
        state["ref"] = torch.where(valid, lp + noise(0.3), 0.0)
        state["out"] = torch.empty(3, device=device)
        state["rewards"] = torch.empty(batch, device=device)
    return state


def _near_logps(x, y, temperature):
    z = x.float() / temperature
    return z.gather(-1, y.clamp(min=0).unsqueeze(-1)).squeeze(-1) - torch.logsumexp(z, -1)


def _prepare_clip(case, g, device, dt):
    shapes = _shapes(case)
    out = _DTYPES[case["out"]]
    state = {"case": case, "device": device, "norm": torch.empty(3, dtype=torch.float64, device=device)}
    n = _elements(case)
    if case["op"] == "clip":
        state["grads"] = [torch.empty(s, dtype=dt, device=device).normal_(0.0, 1e-2, generator=g) for s in shapes]
        state["flat"] = torch.empty(n, dtype=out, device=device)
        state["views"] = [v.view(s) for v, s in zip(state["flat"].split([math.prod(s) for s in shapes]), shapes)]
    else:
        state["grad"] = torch.empty(n, dtype=dt, device=device).normal_(0.0, 1e-3, generator=g)
        state["momentum"] = torch.empty(n, device=device).normal_(0.0, 3e-4, generator=g)
        state["update"] = torch.empty(n, dtype=out, device=device)
    if own:  # a program with lasting gradient buffers describes them to the library once
        state["list"] = _context(device).tensor_list(state["grads"] if case["op"] == "clip" else [state["grad"]])
        if case["op"] == "clip":
            state["out_list"] = _context(device).tensor_list(state["views"])
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"logps": _own_logps, "logps_grad": _own_logps_grad, "policy": _own_policy, "preference": _own_preference,
                "clip": _own_clip, "clip_momentum": _own_clip_momentum}[op](state)
    return {"logps": _logps, "logps_grad": _logps_grad, "policy": _policy, "preference": _preference, "clip": _clipped,
            "clip_momentum": _clipped_momentum}[op](state)


def _own_logps(s):
    _context(s["device"]).token_logps(s["logits"], s["labels"], s["logps"], temperature=s["case"]["temperature"])
    return {"logps": s["logps"]}


def _own_logps_grad(s):
    ctx, t = _context(s["device"]), s["case"]["temperature"]
    ctx.token_logps(s["logits"], s["labels"], s["logps"], row_stats=s["stats"], temperature=t)
    ctx.token_logps_backward(s["logits"], s["labels"], s["stats"], s["grad_logps"], s["grad"], temperature=t)
    return {"logps": s["logps"], "grad": s["grad"]}


def _own_policy(s):
    c = s["case"]
    _context(s["device"]).policy_loss(s["logits"], s["labels"], s["advantages"], s["out"], old_logps=s["old"], ref_logps=s["ref"],
                                      logps=s["logps"], grad_logits=s["grad"], clip_low=0.2, clip_high=0.28, kl_coef=c["kl"],
                                      reduce=c["reduce"], temperature=c["temperature"])
    return {"out": s["out"], "logps": s["logps"], "grad": s["grad"]}


def _own_preference(s):
    c = s["case"]
    _context(s["device"]).preference_loss(s["logits"], s["labels"], s["ref"], s["out"], rewards=s["rewards"], logps=s["logps"],
                                          grad_logits=s["grad"], kind=c["kind"], beta=c["beta"], label_smoothing=c["smoothing"],
                                          average=c["average"], temperature=c["temperature"])
    return {"out": s["out"], "rewards": s["rewards"], "logps": s["logps"], "grad": s["grad"]}


def _own_clip(s):
    _context(s["device"]).clip_grads(s["list"], s["norm"], max_norm=s["case"]["max_norm"], out=s["out_list"])
    return {"norm": s["norm"], "grads": s["flat"]}


def _own_clip_momentum(s):
    ctx = _context(s["device"])
    ctx.grad_norm(s["list"], s["norm"], max_norm=s["case"]["max_norm"])
    ctx.momentum_update(s["grad"], s["momentum"], s["update"], beta=0.95, nesterov=True, grad_scale=s["norm"])
    return {"norm": s["norm"], "momentum": s["momentum"], "update": s["update"]}


def _rows(s):
    """Of every token: its log-probability (64 bits: differences of these follow), the row's softmax, and whether it counts."""
    z = s["logits"].float()
    if s["case"]["temperature"] != 1.0:
        z = z / s["case"]["temperature"]
    valid = s["labels"] >= 0
    at = s["labels"].clamp(min=0).unsqueeze(-1)
    top = z.amax(-1, keepdim=True)
    p = (z - top).exp_()
    total = p.sum(-1, keepdim=True)
    lp = (z.gather(-1, at) - top).double() - total.double().log()
    return torch.where(valid, lp.squeeze(-1), 0.0), p.div_(total), valid, at


def _back(s, p, at, g):
    """The gradient of the logits from that of the log-probabilities."""
    g = (g / s["case"]["temperature"]).float().unsqueeze(-1)
    return p.mul_(-g).scatter_add_(-1, at, g).to(s["logits"].dtype)


def _logps(s):
    return {"logps": _rows(s)[0].float()}


def _logps_grad(s):
    lp, p, valid, at = _rows(s)
    return {"logps": lp.float(), "grad": _back(s, p, at, torch.where(valid, s["grad_logps"], 0.0))}


def _policy(s):
    c = s["case"]
    lp, p, valid, at = _rows(s)
    counts = valid.sum(-1, keepdim=True).clamp(min=1).double()
    weight = {"token": 1.0 / valid.sum().clamp(min=1).double(), "sequence": 1.0 / (counts * c["batch"]),
              "sum": torch.ones_like(counts)}[c["reduce"]]
    weight = torch.where(valid, weight, 0.0)
    a = s["advantages"].double() if c["per_token"] else s["advantages"].double().unsqueeze(-1)
    ratio = (lp - s["old"].double()).exp() if c["old"] else torch.ones_like(lp)
    free, held = -a * ratio, -a * ratio.clamp(1.0 - 0.2, 1.0 + 0.28)
    term = torch.maximum(free, held)
    g = torch.where(free >= held, free, 0.0)
    kl = torch.zeros_like(lp)
    if c["kl"]:
        e = torch.where(valid, s["ref"].double() - lp, 0.0)
        kl = torch.expm1(e) - e
        g = g - c["kl"] * torch.expm1(e)
    sums = [(weight * v).sum() for v in (term + c["kl"] * kl, term, kl, (held > free).double())]
    return {"out": torch.stack(sums).float(), "logps": lp.float(), "grad": _back(s, p, at, weight * g)}


def _preference(s):
    c = s["case"]
    lp, p, valid, at = _rows(s)
    pairs = c["batch"] // 2
    part = torch.where(valid, 1.0, 0.0).double()
    if c["average"]:
        part = part / valid.sum(-1, keepdim=True).clamp(min=1)
    score = (part * (lp - s["ref"].double())).sum(-1)
    margin = score[:pairs] - score[pairs:]
    h = c["beta"] * margin
    if c["kind"] == "sigmoid":
        eps = c["smoothing"]
        loss = (1 - eps) * (1 + (-h).exp()).log() + eps * (1 + h.exp()).log()
        d = c["beta"] * (eps / (1 + (-h).exp()) - (1 - eps) / (1 + h.exp()))
    else:
        off = margin - 1.0 / (2.0 * c["beta"])
        loss, d = off * off, 2.0 * off
    g = torch.cat([d, -d]).unsqueeze(-1) / pairs * part
    out = torch.stack([loss.mean(), h.mean(), (margin > 0).double().mean()]).float()
    return {"out": out, "rewards": (c["beta"] * score).float(), "logps": lp.float(), "grad": _back(s, p, at, g)}


def _norm(tensors, max_norm):
    total = torch.stack([t.double().square().sum() for t in tensors]).sum()
    norm = total.sqrt()
    return torch.stack([total, norm, (max_norm / (norm + 1e-6)).clamp(max=1.0)])


def _clipped(s):
    norm = _norm(s["grads"], s["case"]["max_norm"])
    coef, out = norm[2].float(), _DTYPES[s["case"]["out"]]
    return {"norm": norm, "grads": torch.cat([(t.float() * coef).to(out).reshape(-1) for t in s["grads"]])}


def _clipped_momentum(s):
    norm = _norm([s["grad"]], s["case"]["max_norm"])
    t = (s["grad"].float() * norm[2].float()) * (1.0 - 0.95)
    s["momentum"].mul_(0.95).add_(t)
    return {"norm": norm, "momentum": s["momentum"], "update": (t + 0.95 * s["momentum"]).to(s["update"].dtype)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("clip"):
        return _exact_clip(case, s)
    x, y, t = s["logits"], s["labels"], case["temperature"]
    chosen = y.clamp(min=0)
    pick = [torch.log_softmax(x[b].double() / t, -1).gather(-1, chosen[b][:, None])[:, 0] for b in range(case["batch"])]
    lp = torch.stack(pick)
    lp[y < 0] = 0.0
    if case["op"] == "logps":
        return {"logps": lp}
    n = (y >= 0).sum(1)
    answer = {"logps": lp}
    if case["op"] == "logps_grad":
        g = s["grad_logps"].double() * (y >= 0)
    elif case["op"] == "policy":
        w = (y >= 0).double()
        if case["reduce"] == "token":
            w = w / max(1, int(n.sum()))
        elif case["reduce"] == "sequence":
            w = w / n.clamp(min=1)[:, None] / case["batch"]
        lp_ = lp.clone().requires_grad_()
        a = s["advantages"].double().reshape(case["batch"], -1)
        r = torch.exp(lp_ - s["old"].double()) if case["old"] else torch.exp(lp_ - lp)
        inside = torch.minimum(torch.maximum(r, torch.tensor(0.8, dtype=r.dtype, device=r.device)),
                               torch.tensor(1.28, dtype=r.dtype, device=r.device))
        pg = -torch.minimum(a * r, a * inside)
        e = (s["ref"].double() - lp_) if case["kl"] else 0.0 * lp_
        kl = torch.expm1(e) - e
        loss = (w * (pg + case["kl"] * kl)).sum()
        g, = torch.autograd.grad(loss, lp_)
        g = torch.where(w > 0, g, 0.0)
        answer["out"] = torch.stack([loss, (w * pg).sum(), (w * kl).sum(), (w * (a * inside < a * r)).sum()]).detach()
    else:
        w = (y >= 0).double()
        if case["average"]:
            w = w / n.clamp(min=1)[:, None]
        lp_ = lp.clone().requires_grad_()
        score = (w * (lp_ - s["ref"].double())).sum(1)
        won, lost = score.chunk(2)
        if case["kind"] == "sigmoid":
            ls = torch.nn.functional.logsigmoid
            h = case["beta"] * (won - lost)
            loss = -((1 - case["smoothing"]) * ls(h) + case["smoothing"] * ls(-h)).mean()
        else:
            loss = ((won - lost - 0.5 / case["beta"]) ** 2).mean()
        g, = torch.autograd.grad(loss, lp_)
        answer["out"] = torch.stack([loss, case["beta"] * (won - lost).mean(), (won > lost).double().mean()]).detach()
        answer["rewards"] = (case["beta"] * score).detach()
    grads = []
    for b in range(case["batch"]):
        d = torch.softmax(x[b].double() / t, -1)
        d.scatter_add_(-1, chosen[b][:, None], torch.full_like(d[:, :1], -1.0))
        grads.append(d.mul_(-g[b][:, None] / t))
    answer["grad"] = torch.stack(grads)
    return answer


def _exact_clip(case, s):
    every = torch.cat([t.reshape(-1) for t in s["grads"]]) if case["op"] == "clip" else s["grad"]
    every = every.double()
    size = torch.linalg.vector_norm(every)
    coef = torch.minimum(torch.ones_like(size), case["max_norm"] / (size + 1e-6))
    norm = torch.stack([size * size, size, coef])
    if case["op"] == "clip":
        return {"norm": norm, "grads": every.mul_(coef)}
    step = every.mul_(coef * 0.05)
    m = s["momentum"].double().mul_(0.95).add_(step)
    return {"norm": norm, "momentum": m, "update": step.add_(m, alpha=0.95)}
