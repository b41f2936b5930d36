"""Operators around the layers whose weights the step moves, as they are measured: activations kept in 8 bits, products
in 8-bit integers, the gradients formed out of what was kept, and the verification of drafted tokens.

A case is one call (or the calls that belong together) at one size.  With `own` false run() computes the plain form in
elementary torch operations; with `own` true it calls the library.  A linear layer is y = x w^T: x [tokens, k],
w [n, k], y [tokens, n].  8-bit rows are integers with a scale per row (a token's activations, an output channel's
weights), their storage padded to rows of whole 16 bytes."""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_WORKSPACE = 512 << 20
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
def _checkpoint(name, dtype, tokens, k):
    return {"name": name, "op": "checkpoint", "dtype": dtype, "tokens": tokens, "k": k}


def _linear(name, dtype, out, tokens, n, k):
    return {"name": name, "op": "linear", "dtype": dtype, "out": out, "tokens": tokens, "n": n, "k": k}


def _backward(name, out, accumulate, tokens, n, k):
    return {"name": name, "op": "backward", "out": out, "accumulate": accumulate, "tokens": tokens, "n": n, "k": k}


def _verify(name, dtype, batch, draft, vocab, **more):
    case = {"name": name, "op": "verify", "dtype": dtype, "batch": batch, "draft": draft, "vocab": vocab,
            "draft_logits": True, "temperature": 1.0, "ragged": 0, "noise": 0.7}
    case.update(more)
    return case


def listed():
    return [
        # what a test model keeps of a short sequence, single precision, rows of an odd length
        _checkpoint("keep short sequence", "f32", 37, 1101),
        # the input of a down projection over a training batch, kept and read back
        _checkpoint("keep layer input", "bf16", 8192, 9728),
        # one token through an up projection: a call whose latency counts
        _linear("one token", "bf16", "bf16", 1, 9728, 2560),
        # the next scores of thirteen sequences over a full vocabulary: the weights are read once
        _linear("head of thirteen sequences", "bf16", "f32", 13, 151936, 2560),
        # an odd test model in single precision
        _linear("odd layer", "f32", "f32", 333, 1001, 1237),
        # a training batch through an up projection
        _linear("training batch", "bf16", "bf16", 8192, 9728, 2560),
        # both gradients of a test model's layer
        _backward("gradients of odd layer", "bf16", False, 61, 301, 1237),
        # a query projection, gradients in the dtype the step reads
        _backward("gradients of query projection", "bf16", False, 2048, 4096, 2560),
        # an up projection, the weights' gradient accumulated in single precision over micro-batches
        _backward("gradients accumulated", "f32", True, 8192, 9728, 2560),
        # one sequence of a test model, four drafted tokens
        _verify("one sequence", "f32", 1, 4, 1000),
        # drafts looked up in the prompt, without probabilities of their own, of different lengths
        _verify("looked up drafts", "bf16", 8, 7, 50257, draft_logits=False, temperature=0.8, ragged=3),
        # a batch of sampled answers with a draft model
        _verify("batch with draft model", "bf16", 32, 5, 151936, ragged=2),
    ]


_MOST = 8192 * 9728 * 2560  # products of the largest listed layer
_MOST_ROWS = 32 * 11 * 151936 * 2  # bytes of scores of the largest listed verification


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _size(rng, low, high):
    """Some sizes are multiples of 64, as most layers' are, the others anything."""
    n = _log_int(rng, low, high)
    return min(high, (n + 63) // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["checkpoint", "linear", "linear", "backward", "backward", "verify", "verify"])
    dtype, out = rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"])
    if op == "checkpoint":
        case = _checkpoint("", dtype, _log_int(rng, 1, 8192), _size(rng, 16, 9728))
    elif op == "verify":
        vocab, draft, batch = _log_int(rng, 300, 151936), rng.randrange(1, 9), _log_int(rng, 1, 64)
        while batch * (2 * draft + 1) * vocab * (2 if dtype == "bf16" else 4) > _MOST_ROWS:
            batch = max(1, batch // 2)
        case = _verify("", dtype, batch, draft, vocab, draft_logits=rng.random() < 0.7,
                       temperature=rng.choice([1.0, round(rng.uniform(0.4, 1.5), 2), 0.0]), ragged=rng.randrange(0, draft + 1),
                       noise=round(rng.uniform(0.2, 1.5), 2))
    else:
        tokens, n, k = _log_int(rng, 1, 8192), _size(rng, 40, 9728), _size(rng, 40, 9728)
        if op == "linear" and rng.random() < 0.2:
            tokens, n = min(tokens, 32), _size(rng, 9728, 151936)
        while tokens * n * k > _MOST:
            tokens = tokens // 2
        case = _linear("", dtype, out, tokens, n, k) if op == "linear" else _backward("", out, rng.random() < 0.4, tokens, n, k)
    del case["name"]
    return case


def work(case):
    if case["op"] == "checkpoint":
        # in, the integers and scales out and in again, the values out
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["tokens"] * (case["k"] * (2 * e + 2) + 8), "flops": 4 * case["tokens"] * case["k"]}
    if case["op"] == "verify":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = case["batch"] * (2 * case["draft"] + 1 if case["draft_logits"] and case["temperature"] else case["draft"] + 1)
        return {"bytes": rows * case["vocab"] * e + case["batch"] * (case["draft"] + 1) * 32, "flops": 5 * rows * case["vocab"]}
    t, n, k = case["tokens"], case["n"], case["k"]
    eo = 2 if case["out"] == "bf16" else 4
    if case["op"] == "linear":
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": t * k * e + n * (k + 4) + t * n * eo, "flops": 2 * t * n * k}
    # gradient of y, integers of x and w, gradients of x and w
    return {"bytes": t * n * 2 + (t + n) * (k + 4) + t * k * 2 + n * k * eo * (2 if case["accumulate"] else 1),
            "flops": 4 * t * n * k}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _padded(rows, cols, device):
    """8-bit rows at addresses of whole 16 bytes."""
    return torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8, device=device)[:, :cols]


def _rounded(x):
    """Integers and scales of the rows of x."""
    top = x.abs().amax(-1).float()
    scale = (top.double() / 127).float()
    q = torch.round(x.double() / torch.where(scale > 0, scale, 1.0).double().unsqueeze(-1))
    return q.clamp(-127, 127).to(torch.int8), scale


def _activations(g, device, tokens, k, dtype):
    """Activations with a few large channels, as layers have them."""
    x = torch.empty(tokens, k, device=device).normal_(0.0, 1.0, generator=g)
    x *= torch.empty(k, device=device).normal_(0.0, 0.6, generator=g).exp_()
    return x.to(dtype)


def _eight(x):
    q = _padded(x.shape[0], x.shape[1], x.device)
    scale = torch.empty(x.shape[0], device=x.device)
    for i in range(0, x.shape[0], 8192):
        q[i:i + 8192], scale[i:i + 8192] = _rounded(x[i:i + 8192])
    return q, scale


def _weights(g, device, n, k):
    return _eight(torch.empty(n, k, device=device).normal_(0.0, k ** -0.5, generator=g))


def prepare(case, seed):
    device = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=device).manual_seed(seed * 7919 + 29)
    state = {"case": case, "device": device}
    op = case["op"]
    if op == "verify":
        return _prepare_verify(case, g, device, state)
    t, k = case["tokens"], case["k"]
    if op == "checkpoint":
        state["x"] = _activations(g, device, t, k, _DTYPES[case["dtype"]])
        state["q"], state["scale"] = _padded(t, k, device), torch.empty(t, device=device)
        state["values"] = torch.empty_like(state["x"])
    elif op == "linear":
        state["x"] = _activations(g, device, t, k, _DTYPES[case["dtype"]])
        state["w"] = _weights(g, device, case["n"], k)
        state["y"] = torch.empty(t, case["n"], dtype=_DTYPES[case["out"]], device=device)
    else:
        n = case["n"]
        state["x8"] = _eight(_activations(g, device, t, k, torch.bfloat16))
        state["w"] = _weights(g, device, n, k)
        state["grad_y"] = torch.empty(t, n, device=device).normal_(0.0, 1e-3, generator=g).to(torch.bfloat16)
        state["grad_x"] = torch.empty(t, k, dtype=torch.bfloat16, device=device)
        state["grad_w"] = torch.empty(n, k, device=device).normal_(0.0, 1e-3, generator=g).to(_DTYPES[case["out"]])
    if own:  # a program keeps what describes its lasting buffers
        from newton_schulz_amd import Rows8
        if op == "checkpoint":
            state["kept"] = Rows8(state["q"], state["scale"])
        else:
            state["w8"] = Rows8(*state["w"])
            if op == "backward":
                state["kept"] = Rows8(*state["x8"])
    return state


def _prepare_verify(case, g, device, state):
    b, d, v = case["batch"], case["draft"], case["vocab"]
    dt = _DTYPES[case["dtype"]]
    logits = torch.empty(b, d + 1, v, device=device).normal_(0.0, 2.0, generator=g)
    # answers have a handful of likely tokens at each place
    likely = torch.randint(v, (b, d + 1, 8), generator=g, device=device)
    logits.scatter_add_(-1, likely, torch.rand(b, d + 1, 8, generator=g, device=device) * 10.0 + 3.0)
    near = logits[:, :d] + case["noise"] * torch.empty(b, d, v, device=device).normal_(0.0, 1.0, generator=g)
    logits, near = logits.to(dt), near.to(dt)
    # the draft model samples at the same temperature (a deterministic draft takes its most likely token)
    z = near.float()
    if case["draft_logits"] and case["temperature"]:
        z = z / case["temperature"] - torch.log(torch.empty_like(z).exponential_(1.0, generator=g))
    tokens = z.argmax(-1)
    # sequences near their end draft fewer tokens
    length = torch.tensor([d - (i * case["ragged"]) % (d + 1) for i in range(b)], device=device)
    tokens.masked_fill_(torch.arange(d, device=device) >= length.unsqueeze(-1), -1)
    state.update(logits=logits, near=near if case["draft_logits"] else None, draft=tokens,
                 uniforms=torch.rand(b, d + 1, generator=g, device=device),
                 tokens=torch.empty(b, d + 1, dtype=torch.int64, device=device),
                 accepted=torch.empty(b, dtype=torch.int64, device=device), logps=torch.empty(b, d + 1, device=device))
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"checkpoint": _own_checkpoint, "linear": _own_linear, "backward": _own_backward, "verify": _own_verify}[op](state)
    return {"checkpoint": _plain_checkpoint, "linear": _plain_linear, "backward": _plain_backward, "verify": _plain_verify}[op](state)


def _own_checkpoint(s):
    ctx = _context(s["device"])
    ctx.quantize_rows(s["x"], s["kept"])
    ctx.dequantize_rows(s["kept"], s["values"])
    return {"scale": s["scale"], "values": s["values"]}


def _own_linear(s):
    _context(s["device"]).linear8(s["x"], s["w8"], s["y"])
    return {"y": s["y"]}


def _own_backward(s):
    ctx = _context(s["device"])
    ctx.input_grad8(s["grad_y"], s["w8"], s["grad_x"])
    ctx.weight_grad8(s["grad_y"], s["kept"], s["grad_w"], accumulate=s["case"]["accumulate"])
    return {"grad_x": s["grad_x"], "grad_w": s["grad_w"]}


def _own_verify(s):
    _context(s["device"]).verify_draft(s["logits"], s["draft"], s["tokens"], s["accepted"], draft_logits=s["near"],
                                       uniforms=s["uniforms"], logps=s["logps"], temperature=s["case"]["temperature"])
    return {"tokens": s["tokens"], "accepted": s["accepted"], "logps": s["logps"]}


def _plain_checkpoint(s):
    q, scale = _rounded(s["x"])
    return {"scale": scale, "values": (q.float() * scale.unsqueeze(-1)).to(s["x"].dtype)}


def _plain_linear(s):
    q, scale = _rounded(s["x"])
    w, w_scale = s["w"]
    return {"y": ((q.float() @ w.float().t()) * scale.unsqueeze(-1) * w_scale).to(s["y"].dtype)}


def _plain_backward(s):
    g = s["grad_y"].float()
    (q, scale), (w, w_scale) = s["x8"], s["w"]
    grad_x = g @ (w.float() * w_scale.unsqueeze(-1))
    grad_w = g.t() @ (q.float() * scale.unsqueeze(-1))
    if s["case"]["accumulate"]:
        grad_w = grad_w + s["grad_w"].float()
    s["grad_w"].copy_(grad_w)
    return {"grad_x": grad_x.to(torch.bfloat16), "grad_w": s["grad_w"]}


def _plain_verify(s):
    c, draft, x = s["case"], s["draft"], s["logits"]
    b, d, v = c["batch"], c["draft"], c["vocab"]
    greedy = c["temperature"] == 0
    t = 1.0 if greedy else c["temperature"]
    valid = draft >= 0
    at = draft.clamp(min=0).unsqueeze(-1)

    def log_sums(z):
        """Of every row the logarithm of the sum of exp(z / t), 32-bit exponentials added in 64."""
        top = z.amax(-1, keepdim=True).float()
        return (top.double() / t).squeeze(-1) + torch.exp((z.float() - top) / t).sum(-1, dtype=torch.float64).log()

    def log_probs(z, sums):
        return z.gather(-1, at).squeeze(-1).double() / t - sums

    sums = log_sums(x)
    with_draft = s["near"] is not None and not greedy
    if greedy:
        best = x.argmax(-1)
        taken = valid & (best[:, :d] == draft)
    else:
        own_p = log_probs(x[:, :d], sums[:, :d]).exp()
        near_p = log_probs(s["near"], log_sums(s["near"])).exp() if with_draft else torch.ones_like(own_p)
        taken = valid & (s["uniforms"][:, :d].double() * near_p < own_p)
    accepted = taken.long().cumprod(-1).sum(-1)
    # the distribution of the token behind the accepted ones, in 64 bits
    each = torch.arange(b, device=x.device)
    if greedy:
        chosen = best[each, accepted]
    else:
        p = torch.softmax(x[each, accepted].double() / t, -1)
        place = accepted.clamp(max=d - 1)
        drafted = (accepted < d) & valid[each, place]
        if with_draft:
            q = torch.softmax(s["near"][each, place].double() / t, -1)
        else:
            q = torch.zeros_like(p).scatter_(-1, at[each, place], 1.0)
        left = torch.where(drafted.unsqueeze(-1), (p - q).clamp(min=0), p)
        left = torch.where(left.sum(-1, keepdim=True) > 0, left, p)
        run_of = left.cumsum(-1)
        above = (run_of > s["uniforms"][:, d:].double() * run_of[:, -1:]) & (left > 0)
        last = v - 1 - (left > 0).flip(-1).long().argmax(-1)
        chosen = torch.where(above.any(-1), above.long().argmax(-1), last)
    places = torch.arange(d + 1, device=x.device)
    padded = torch.cat([draft, torch.full_like(draft[:, :1], -1)], 1)
    tokens = torch.where(places < accepted.unsqueeze(-1), padded, -1)
    tokens[each, accepted] = chosen
    logps = x.gather(-1, tokens.clamp(min=0).unsqueeze(-1)).squeeze(-1).double() / t - sums
    return {"tokens": tokens, "accepted": accepted, "logps": torch.where(tokens >= 0, logps, 0.0).float()}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(x):
    """Values of 8-bit rows: each the nearest multiple of its row's scale."""
    x = x.double()
    scale = (x.abs().max(dim=1).values / 127.0).to(torch.float32).double()
    steps = torch.where(scale[:, None] > 0, x / scale[:, None], torch.zeros_like(x))
    return steps.round_().clamp_(-127, 127), scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "checkpoint":
        q, scale = _exact_rows(s["x"])
        return {"scale": scale, "values": q.mul_(scale[:, None])}
    if case["op"] == "linear":
        q, scale = _exact_rows(s["x"])
        w, w_scale = s["w"]
        y = torch.matmul(q, w.double().t())
        return {"y": y.mul_(torch.outer(scale, w_scale.double()))}
    if case["op"] == "backward":
        g = s["grad_y"].double()
        x, w = (q.double().mul_(scale.double()[:, None]) for q, scale in (s["x8"], s["w"]))
        grad_w = torch.matmul(g.t(), x)
        return {"grad_x": torch.matmul(g, w), "grad_w": grad_w.add_(s["grad_w"].double()) if case["accumulate"] else grad_w}
    tokens, logps, counts = [], [], []
    u, draft = s["uniforms"].double().cpu(), s["draft"].cpu()
    t = case["temperature"] or 1.0
    for b in range(case["batch"]):
        row, lp, i = [], [], 0
        while True:
            z = torch.log_softmax(s["logits"][b, i].double() / t, -1)
            y = int(draft[b, i]) if i < case["draft"] else -1
            if case["temperature"] == 0:
                best = int((z == z.max()).nonzero()[0])
                row.append(best)
                lp.append(float(z[best]))
                if best != y:
                    break
                i += 1
                continue
            near = None
            if y >= 0 and s["near"] is not None:
                near = torch.softmax(s["near"][b, i].double() / t, -1)
            if y >= 0 and float(u[b, i]) * (1.0 if near is None else float(near[y])) < math.exp(float(z[y])):
                row.append(y)
                lp.append(float(z[y]))
                i += 1
                continue
            weights = z.exp()
            if y >= 0:
                rest = weights.clone()
                if near is None:
                    rest[y] = 0.0
                else:
                    rest = torch.relu(rest - near)
                weights = rest if float(rest.sum()) > 0 else weights
            edges = weights.cumsum(0)
            inside = ((edges > float(u[b, -1]) * float(edges[-1])) & (weights > 0)).nonzero()
            pick = int(inside[0]) if len(inside) else int(weights.nonzero()[-1])
            row.append(pick)
            lp.append(float(z[pick]))
            break
        counts.append(len(row) - 1)
        fill = case["draft"] + 1 - len(row)
        tokens.append(row + [-1] * fill)
        logps.append(lp + [0.0] * fill)
    return {"tokens": torch.tensor(tokens, device=s["device"]), "accepted": torch.tensor(counts, device=s["device"]),
            "logps": torch.tensor(logps, dtype=torch.float64, device=s["device"])}
