"""Log-probabilities, policy and preference loss with their gradients against
the binary64 oracle (needs a gfx950 GPU).

Tolerances, with u = 2^-24 (half a binary32 step, relative):
  * S = sum_v exp(z_v - M).  A term's argument has at most three roundings
    (subtraction, the constant log2 e / T, the product; the constant is rounded up
    in some places of 16 bytes and down in others, with their mean within u / 4),
    so its relative error on average is 3 u |z_v - M| and 2 u of the exponential; averaged with the softmax,
    E[M - z] <= entropy <= log V.  Sums of at most n terms per thread and the
    joins add at most (n + n / 4 * 3 + 40) u: a rescale (product, exponential)
    for every 16 bytes of scores, 40 for the joins across threads.
    So log S is off by at most s = u (3 log V + 2 + 1.75 n + 40), and the
    label's own score by 2 u |z_y - M| (subtraction; the rest is binary64).
  * lp is stored in binary32: u |lp| more.
  * a gradient G ([v = y] - p_v): p_v is off by p_v (s + u (3 |z_v - M| + 8)),
    the label's sum rounds once more, and storing rounds by half a step.
n is counted for a workgroup of 256 threads on a row, 64 below 4096 scores.
"""
import numpy as np
import pytest
import torch

from newton_schulz_amd import Context, MuonError, loss_workspace_bytes
from oracle import loss_oracle as lo

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    c = Context(DEV, 8 << 20)
    yield c
    c.close()


def sum_error(vocab):
    n = -(-vocab // (64 if vocab <= 4096 else 256))
    return U * (3 * np.log(max(vocab, 2)) + 2 + 1.75 * n + 40)


def lp_tolerance(x, y, lp, t):
    """Error of lp before it is stored, per token."""
    z = x / t
    top = np.max(np.where(np.isfinite(z), z, -1e30), -1)
    zy = np.take_along_axis(z, np.clip(y, 0, x.shape[-1] - 1)[..., None], -1)[..., 0]
    off = np.where(np.isfinite(zy), np.abs(zy - top), 0.0)
    return sum_error(x.shape[-1]) + 2 * U * off


def same(got, want, tol, what):
    """NaN and infinities in the same places, the rest within tol."""
    got = got.astype(np.float64)
    odd = ~np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(got[odd & ~np.isnan(want)], want[odd & ~np.isnan(want)]), what
    d = np.abs(got - want)[~odd]
    over = d - np.broadcast_to(tol, want.shape)[~odd]
    assert d.size == 0 or over.max() <= 0, f"{what}: off by {d.max():.3e}, {over.max():.3e} over the tolerance"


def grad_tolerance(x, y, coef, t, want, eps):
    """coef: the gradient in lp, per token; eps: the stored type's step."""
    z = x / t
    p = lo.softmax_ref(x, t)
    off = z.max(-1, keepdims=True) - z
    off = np.where(np.isfinite(off), off, 0.0)
    G = np.abs(coef / t)[..., None]
    arithmetic = G * p * (sum_error(x.shape[-1]) + U * (3 * off + 8)) + 4 * U * G * (np.arange(x.shape[-1]) == y[..., None])
    return arithmetic * (1 + eps) + np.abs(want) * eps / 2 + 1e-37


def make(batch, seq, vocab, dtype, seed=0, pad=0, shift=False, empty=0.3, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    full = torch.randn(batch, seq + int(shift), vocab + pad, generator=g).mul_(scale).to(dtype)
    labels = torch.randint(vocab, (batch, seq), generator=g)
    labels[torch.rand(batch, seq, generator=g) < empty] = -100
    dev = full.to(DEV)[:, :seq, :vocab]
    return dev, labels.to(DEV), full[:, :seq, :vocab].double().numpy(), labels.numpy()


SHAPES = [
    # batch, seq, vocab, pad, shift
    (1, 1, 1, 0, False), (1, 3, 2, 0, False), (2, 5, 7, 0, False), (2, 5, 8, 1, True), (3, 2, 9, 0, False),
    (2, 3, 63, 2, False), (1, 9, 64, 0, True), (2, 2, 65, 0, False), (1, 4, 257, 3, False), (2, 7, 1000, 0, True),
    (3, 11, 4099, 0, False), (1, 2, 16384, 8, False), (2, 40, 5003, 1, True), (1, 600, 513, 0, False),
    (1, 3, 50257, 0, False), (1, 2, 151936, 0, False), (1, 1, 131071, 0, False), (2, 1, 200003, 0, False),
    (1, 300, 33000, 0, False), (1, 270, 20011, 5, False),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("t", [1.0, 0.7])
def test_logps_and_their_gradient(ctx, shape, dtype, t):
    batch, seq, vocab, pad, shift = shape
    x, y, xn, yn = make(batch, seq, vocab, dtype, seed=vocab, pad=pad, shift=shift)
    t32 = t
    logps = torch.full((batch, seq), 7.0, device=DEV)
    stats = torch.empty(batch, seq, 2, device=DEV)
    ctx.token_logps(x, y, logps, row_stats=stats, temperature=t)
    alone = torch.empty_like(logps)
    ctx.token_logps(x, y, alone, temperature=t)
    want = lo.token_logps_ref(xn, yn, t32)
    tol = lp_tolerance(xn, yn, want, t32)
    same(logps.cpu().numpy(), want, tol + U * np.abs(want), "logps")
    assert torch.equal(alone, logps)
    coef = torch.randn(batch, seq, generator=torch.Generator().manual_seed(1)).to(DEV)
    keep = torch.full((batch, seq, vocab + 3), 5.0, dtype=dtype, device=DEV)
    grad = keep[:, :, 1:vocab + 1]  # rows of another stride, at odd addresses
    ctx.token_logps_backward(x, y, stats, coef, grad, temperature=t)
    cn = coef.cpu().double().numpy()
    gw = lo.logits_grad_ref(xn, yn, cn, t32)
    same(grad.float().cpu().numpy(), gw, grad_tolerance(xn, yn, cn, t32, gw, torch.finfo(dtype).eps), "gradient")
    assert (keep[:, :, 0] == 5).all() and (keep[:, :, vocab + 1:] == 5).all()  # nothing beside the rows
    # in place
    own = x.clone()
    ctx.token_logps_backward(own, y, stats, coef, own, temperature=t)
    assert torch.equal(own, grad)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_special_rows(ctx, dtype):
    vocab, low = 1003, torch.finfo(dtype).min
    x, y, _, _ = make(1, 12, vocab, dtype, empty=0.0, seed=5)
    x = x.clone()
    inf = float("inf")
    x[0, 0, 1::2] = -inf            # half the vocabulary masked
    x[0, 1] = -inf                  # nothing left: NaN
    x[0, 2, 1:] = -inf              # one score left
    x[0, 3] = low                   # masks of the type's lowest value alone: uniform
    x[0, 4, 500:] = low
    x[0, 5, 17] = inf               # NaN
    x[0, 6, 17] = float("nan")      # NaN
    x[0, 7] = -inf                  # left out, and never read
    x[0, 8] = float("nan")          # left out, and never read
    x[0, 9, :] = 3e38 if dtype == F32 else 2e38
    x[0, 9, 4] = low                # differences beyond the type's range
    x[0, 10] += 1000.0
    y[0, :] = 2
    y[0, 2] = 0
    y[0, 3] = 1002
    y[0, 7:9] = -1
    y[0, 11] = vocab                # names no score: NaN
    xn, yn = x.double().cpu().numpy(), y.cpu().numpy()
    logps, stats = torch.empty(1, 12, device=DEV), torch.empty(1, 12, 2, device=DEV)
    ctx.token_logps(x, y, logps, row_stats=stats)
    want = lo.token_logps_ref(xn, yn)
    assert np.isnan(want[0, [1, 5, 6, 11]]).all() and (want[0, 7:9] == 0).all()
    same(logps.cpu().numpy(), want, lp_tolerance(xn, yn, want, 1.0) + U * np.abs(want), "logps")
    coef, grad = torch.ones(1, 12, device=DEV), torch.empty_like(x)
    ctx.token_logps_backward(x, y, stats, coef, grad)
    cn = coef.double().cpu().numpy()
    gw = lo.logits_grad_ref(xn, yn, cn)
    fine = np.isfinite(want[0]) & (yn[0] >= 0)  # rows left out have to be zeros exactly
    tol = np.zeros_like(gw)
    with np.errstate(all="ignore"):
        tol[:, fine] = grad_tolerance(xn, yn, cn, 1.0, gw, torch.finfo(dtype).eps)[:, fine]
    same(grad.float().cpu().numpy(), gw, tol, "gradient")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [700, 4099, 50257])
def test_tokens_the_policy_is_sure_of(ctx, vocab, dtype):
    """lp close to 0: S = 1 + u.  The largest score gives exactly 1; in its
    piece of 8 (4) scores, three (two) additions round by at most u = 2^-24
    each, and everything else is relative to u: the terms' arguments, the
    exponentials, S - 1 stored once per slice and once per row."""
    x, y, _, _ = make(1, 24, vocab, dtype, empty=0.0, seed=11, scale=1.0)
    x = x.clone()
    lift = torch.linspace(9, 30, 24, device=DEV)
    x[0, torch.arange(24), y[0]] = lift.to(dtype)
    xn, yn = x.double().cpu().numpy(), y.cpu().numpy()
    want = lo.token_logps_ref(xn, yn)
    assert (want < 0).all() and want.min() > -4 and want.max() > -1e-6
    logps, stats = torch.empty(1, 24, device=DEV), torch.empty(1, 24, 2, device=DEV)
    ctx.token_logps(x, y, logps, row_stats=stats)
    tol = 3.5 * U + np.abs(want) * U * (3 * 32 + 20)
    same(logps.cpu().numpy(), want, tol, "logps")
    # the label's gradient, G (1 - p), keeps that too
    grad, coef = torch.empty_like(x), torch.ones(1, 24, device=DEV)
    ctx.token_logps_backward(x, y, stats, coef, grad)
    got = grad[0, torch.arange(24), y[0]].double().cpu().numpy()
    one_minus_p = -np.expm1(want[0])
    assert (np.abs(got - one_minus_p) <= tol[0] * 1.01 + one_minus_p * (torch.finfo(dtype).eps / 2 + 4 * U)).all()
    out, g2 = torch.empty(4, device=DEV), torch.empty_like(x)
    ctx.policy_loss(x, y, torch.full((1,), -1.0, device=DEV), out, grad_logits=g2, reduce="sum")
    got = g2[0, torch.arange(24), y[0]].double().cpu().numpy()
    assert (np.abs(got - one_minus_p) <= tol[0] * 1.01 + one_minus_p * (torch.finfo(dtype).eps / 2 + 4 * U)).all()


@pytest.mark.parametrize("base,step,t", [(1e10, 1024.0, 2000.0), (-3e12, 262144.0, 1e6), (4.5e4, 0.0625, 1.0), (2e4, 0.03125, 0.5)])
def test_scores_of_large_magnitude(ctx, base, step, t):
    """Differences of a few units on top of scores whose product with log2 e / T
    is far from (and close to) the range the gradient's multiply-add takes."""
    rng = np.random.default_rng(8)
    xn = (np.float32(base) + np.float32(step) * rng.integers(-60, 60, (2, 5, 3001)).astype(np.float32)).astype(np.float32)
    x, xn = torch.from_numpy(xn).to(DEV), xn.astype(np.float64)
    y = torch.from_numpy(rng.integers(0, 3001, (2, 5))).to(DEV)
    yn = y.cpu().numpy()
    logps, stats = torch.empty(2, 5, device=DEV), torch.empty(2, 5, 2, device=DEV)
    ctx.token_logps(x, y, logps, row_stats=stats, temperature=t)
    want = lo.token_logps_ref(xn, yn, t)
    same(logps.cpu().numpy(), want, lp_tolerance(xn, yn, want, t) + U * np.abs(want), "logps")
    coef, grad, g2, out = (torch.ones(2, 5, device=DEV), torch.empty_like(x), torch.empty_like(x),
                           torch.empty(4, device=DEV))
    ctx.token_logps_backward(x, y, stats, coef, grad, temperature=t)
    gw = lo.logits_grad_ref(xn, yn, np.ones((2, 5)), t)
    tol = grad_tolerance(xn, yn, np.ones((2, 5)), t, gw, torch.finfo(F32).eps)
    same(grad.cpu().numpy(), gw, tol, "gradient")
    ctx.policy_loss(x, y, torch.full((2,), -1.0, device=DEV), out, grad_logits=g2, reduce="sum", temperature=t)
    same(g2.cpu().numpy(), gw, tol, "policy gradient")


def placed_like(x):
    """A copy of x with its strides and alignment (the order of a row's sum
    goes by where the row starts)."""
    size = x.storage_offset() + sum((n - 1) * st for n, st in zip(x.shape, x.stride())) + 1
    own = torch.empty(size, dtype=x.dtype, device=DEV).as_strided(x.shape, x.stride(), x.storage_offset())
    return own.copy_(x)


POLICY = [
    # batch, seq, vocab, dtype, pad, reduce, per token, kl, ref given, old given, temperature
    (1, 1, 8, F32, 0, "token", False, 0.0, False, False, 1.0),
    (2, 9, 513, F32, 3, "token", False, 0.05, True, True, 0.7),
    (3, 5, 1000, BF, 0, "sequence", True, 0.0, True, True, 1.0),
    (8, 17, 777, BF, 1, "sequence", False, 0.1, True, True, 1.0),
    (2, 3, 50257, BF, 0, "sum", True, 0.1, True, False, 1.0),
    (1, 2, 151936, BF, 0, "token", False, 0.04, True, True, 1.0),
    (2, 200, 4100, BF, 0, "token", True, 0.04, True, True, 1.3),
    (2, 300, 2051, F32, 2, "token", False, 0.04, True, True, 1.0),
    (1, 400, 33001, BF, 0, "sequence", True, 0.04, True, True, 1.0),
    (1, 300, 20011, F32, 1, "token", True, 0.04, True, True, 1.0),
    (1, 270, 152064, BF, 0, "token", True, 0.04, True, True, 1.0),
]


def policy_inputs(case, seed=3):
    batch, seq, vocab, dtype, pad, reduce, per_token, kl, has_ref, has_old, t = case
    x, y, xn, yn = make(batch, seq, vocab, dtype, seed=seed + vocab, pad=pad)
    if batch > 2:
        y[1] = -1  # a sequence with no token
        yn[1] = -1
    t32 = t
    lp = lo.token_logps_ref(xn, yn, t32)
    rng = np.random.default_rng(seed)

    def near(s):
        v = (lp + s * rng.normal(size=lp.shape)).astype(np.float32)
        v[yn < 0] = np.nan  # never read
        return torch.from_numpy(v).to(DEV)

    adv = rng.normal(size=lp.shape if per_token else batch).astype(np.float32)
    if per_token:
        adv[yn < 0] = np.inf
    old, ref = near(0.3) if has_old else None, near(0.4) if has_ref else None
    return x, y, xn, yn, lp, torch.from_numpy(adv).to(DEV), old, ref, t32


@pytest.mark.parametrize("case", POLICY)
def test_policy_loss(ctx, case):
    batch, seq, vocab, dtype, pad, reduce, per_token, kl, has_ref, has_old, t = case
    x, y, xn, yn, lp, adv, old, ref, t32 = policy_inputs(case)
    out, logps, grad = torch.full((4,), 9.0, device=DEV), torch.empty(batch, seq, device=DEV), torch.empty_like(x)
    kw = dict(clip_low=0.2, clip_high=0.28, kl_coef=kl, reduce=reduce, weight=0.5, temperature=t)
    ctx.policy_loss(x, y, adv, out, old_logps=old, ref_logps=ref, logps=logps, grad_logits=grad, **kw)
    an = adv.double().cpu().numpy()
    on, rn = (v.double().cpu().numpy() if v is not None else None for v in (old, ref))
    want, g = lo.policy_ref(lp, yn, an, on, rn, float(np.float32(0.2)), float(np.float32(0.28)), float(np.float32(kl)),
                            reduce, 0.5)
    d = lp_tolerance(xn, yn, lp, t32)
    same(logps.cpu().numpy(), lp, d + U * np.abs(lp), "logps")
    # how far the errors of lp reach: the ratio and exp(e) change by that much of themselves
    valid = yn >= 0
    w = lo.policy_weights(yn, reduce)
    a = np.where(valid, an if per_token else np.broadcast_to(an[:, None], lp.shape), 0.0)
    ratio = np.where(valid, np.exp(lp - on), 1.0) if has_old else np.ones_like(lp)
    if has_old:  # no ratio lies so near a border that the rounding could take it across
        assert min(np.abs(ratio - 0.8)[valid].min(), np.abs(ratio - 1.28)[valid].min()) > 4 * d.max()
    e = np.where(valid, rn - lp, 0.0) if has_ref else np.zeros_like(lp)
    slack = 1.01  # second order
    d_pg = slack * (w * np.abs(a) * ratio * d).sum()
    d_kl = slack * (w * np.abs(np.expm1(e)) * d + w * d * d * np.exp(e)).sum()
    tol = np.array([0.5 * (d_pg + kl * d_kl), d_pg, d_kl, 0.0]) + U * np.abs(want) + 1e-12
    same(out.cpu().numpy(), want, tol, "out")
    d_g = slack * 0.5 * w * (np.abs(a) * ratio + kl * np.exp(e)) * d + U * np.abs(g)
    tol = grad_tolerance(xn, yn, g, t32, lo.logits_grad_ref(xn, yn, g, t32), torch.finfo(dtype).eps)
    onehot = np.arange(vocab) == yn[..., None]
    tol += (1 + torch.finfo(dtype).eps) * (d_g / t32)[..., None] * np.abs(onehot - lo.softmax_ref(xn, t32))
    same(grad.float().cpu().numpy(), lo.logits_grad_ref(xn, yn, g, t32), tol, "gradient")
    # evaluation alone, and in place: the same bits
    again, own = torch.empty_like(out), placed_like(x)
    ctx.policy_loss(x, y, adv, again, old_logps=old, ref_logps=ref, **kw)
    assert torch.equal(again, out)
    ctx.policy_loss(own, y, adv, again, old_logps=old, ref_logps=ref, grad_logits=own, **kw)
    assert torch.equal(again, out) and torch.equal(own, grad)


@pytest.mark.parametrize("case", [c for c in POLICY if c[2] > 4000])
def test_policy_loss_without_waiting(case):
    """No poll at all: workgroups compute what their row's others have not
    published yet, in place too, and nothing changes."""
    batch, seq, vocab, dtype, pad, reduce, per_token, kl, has_ref, has_old, t = case
    x, y, xn, yn, lp, adv, old, ref, t32 = policy_inputs(case)
    kw = dict(old_logps=old, ref_logps=ref, clip_low=0.2, clip_high=0.28, kl_coef=kl, reduce=reduce, temperature=t)
    c = Context(DEV, 8 << 20)
    got = []
    for polls in (1 << 14, 0):
        c.set_loss_polls(polls)
        out, logps, own = torch.empty(4, device=DEV), torch.empty(batch, seq, device=DEV), placed_like(x)
        c.policy_loss(own, y, adv, out, logps=logps, grad_logits=own, **kw)
        got.append((out, logps, own))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    with pytest.raises(MuonError):
        c.set_loss_polls(-1)
    c.close()


PREFERENCE = [
    # pairs, seq, vocab, dtype, pad, kind, smoothing, average, reference
    (1, 1, 9, F32, 0, "sigmoid", 0.0, False, True),
    (3, 33, 411, F32, 2, "sigmoid", 0.1, False, True),
    (2, 7, 50257, BF, 0, "sigmoid", 0.0, True, False),
    (5, 70, 1001, BF, 1, "ipo", 0.0, True, True),
    (2, 150, 4099, BF, 0, "sigmoid", 0.0, False, True),
    (1, 2, 151936, BF, 0, "ipo", 0.0, False, True),
]


@pytest.mark.parametrize("case", PREFERENCE)
def test_preference_loss(ctx, case):
    pairs, seq, vocab, dtype, pad, kind, smoothing, average, has_ref = case
    batch = 2 * pairs
    x, y, xn, yn = make(batch, seq, vocab, dtype, seed=vocab, pad=pad)
    if pairs > 1:
        y[batch - 1] = -1  # a rejected answer with no token
        yn[batch - 1] = -1
    lp = lo.token_logps_ref(xn, yn)
    ref = None
    if has_ref:
        v = (lp + 0.2 * np.random.default_rng(1).normal(size=lp.shape)).astype(np.float32)
        v[yn < 0] = np.inf  # never read
        ref = torch.from_numpy(v).to(DEV)
    rn = ref.double().cpu().numpy() if has_ref else None
    beta = float(np.float32(0.1))
    out, rewards = torch.empty(3, device=DEV), torch.empty(batch, device=DEV)
    logps, grad = torch.empty(batch, seq, device=DEV), torch.empty_like(x)
    kw = dict(kind=kind, beta=0.1, label_smoothing=smoothing, average=average, weight=2.0)
    ctx.preference_loss(x, y, ref, out, rewards=rewards, logps=logps, grad_logits=grad, **kw)
    s32 = float(np.float32(smoothing))
    want, rw, g = lo.preference_ref(lp, yn, rn, kind, beta, s32, average, 2.0)
    d = lp_tolerance(xn, yn, lp, 1.0)
    same(logps.cpu().numpy(), lp, d + U * np.abs(lp), "logps")
    valid = yn >= 0
    n = np.maximum(valid.sum(1), 1) if average else np.ones(batch)
    d_score = np.where(valid, d, 0.0).sum(1) / n + 1e-13
    same(rewards.cpu().numpy(), rw, beta * d_score + U * np.abs(rw), "rewards")
    d_m = d_score[:pairs] + d_score[pairs:]
    m = (rw[:pairs] - rw[pairs:]) / beta
    assert (np.abs(m) > d_m).all()
    if kind == "sigmoid":
        d_loss, d_slope = beta * d_m, beta * beta * d_m / 4
    else:
        d_loss, d_slope = 2 * np.abs(m - 0.5 / beta) * d_m + d_m ** 2, 2 * d_m
    tol = np.array([2 * d_loss.mean(), beta * d_m.mean(), 0.0]) + 2 * U * np.abs(want) + 1e-12
    same(out.cpu().numpy(), want, tol, "out")
    d_g = np.where(valid, (2 / pairs * np.tile(d_slope, 2) / n)[:, None], 0.0) + U * np.abs(g)
    gw = lo.logits_grad_ref(xn, yn, g)
    tol = grad_tolerance(xn, yn, g, 1.0, gw, torch.finfo(dtype).eps)
    onehot = np.arange(vocab) == yn[..., None]
    tol += (1 + torch.finfo(dtype).eps) * d_g[..., None] * np.abs(onehot - lo.softmax_ref(xn))
    same(grad.float().cpu().numpy(), gw, tol, "gradient")
    again, own = torch.empty_like(out), placed_like(x)
    ctx.preference_loss(x, y, ref, again, **kw)
    assert torch.equal(again, out)
    ctx.preference_loss(own, y, ref, again, grad_logits=own, **kw)
    assert torch.equal(again, out) and torch.equal(own, grad)


def test_no_token_and_empty_batches(ctx):
    x, y, _, _ = make(2, 4, 300, BF)
    y.fill_(-100)
    out, grad, logps = torch.full((4,), 3.0, device=DEV), torch.ones_like(x), torch.ones(2, 4, device=DEV)
    for reduce in ("token", "sequence", "sum"):
        ctx.policy_loss(x, y, torch.ones(2, device=DEV), out, logps=logps, grad_logits=grad, reduce=reduce)
        assert (out == 0).all() and (grad == 0).all() and (logps == 0).all()
    out3 = torch.full((3,), 3.0, device=DEV)
    ctx.preference_loss(x, y, None, out3, grad_logits=grad)
    assert out3[0].item() == pytest.approx(np.log(2), abs=1e-7) and (out3[1:] == 0).all() and (grad == 0).all()
    for shape in ((0, 4, 300), (2, 0, 300)):
        e = torch.empty(shape, dtype=BF, device=DEV)
        ye, le = torch.empty(shape[:2], dtype=torch.int64, device=DEV), torch.empty(shape[:2], device=DEV)
        ctx.token_logps(e, ye, le)
        out.fill_(3.0)
        ctx.policy_loss(e, ye, torch.empty(shape[0], device=DEV), out, logps=le, grad_logits=torch.empty_like(e))
        assert (out == 0).all()
        ctx.preference_loss(e, ye, None, out3, grad_logits=torch.empty_like(e))
        assert out3[0].item() == pytest.approx(np.log(2) if shape[0] else 0.0, abs=1e-7)


def test_rows_beyond_32_bit_offsets(ctx):
    """Two sequences 5 GB apart in one buffer, scores and gradient alike."""
    stride, seq, vocab = 2_500_000_003, 3, 1001
    buf = torch.zeros(stride + seq * vocab, dtype=BF, device=DEV)
    x = buf.as_strided((2, seq, vocab), (stride, vocab, 1))
    small, y, xn, yn = make(2, seq, vocab, BF, empty=0.0)
    x.copy_(small)
    logps, out = torch.empty(2, seq, device=DEV), torch.empty(4, device=DEV)
    ctx.policy_loss(x, y, torch.ones(2, device=DEV), out, logps=logps, grad_logits=x)
    grad, out2 = torch.empty_like(small), torch.empty(4, device=DEV)
    ctx.policy_loss(small, y, torch.ones(2, device=DEV), out2, grad_logits=grad)
    want = lo.token_logps_ref(xn, yn)
    same(logps.cpu().numpy(), want, lp_tolerance(xn, yn, want, 1.0) + U * np.abs(want), "logps")
    assert torch.equal(x, grad) and torch.equal(out, out2)


def test_broadcast_and_sequence_major_scores(ctx):
    """One row for every token (strides 0), and [seq, batch] storage."""
    base, _, bn, _ = make(1, 1, 777, F32)
    x = base.expand(2, 3, 777)
    y = torch.tensor([[1, 5, -1], [776, 0, 9]], device=DEV)
    yn, xn = y.cpu().numpy(), np.broadcast_to(bn, (2, 3, 777))
    logps, stats = torch.empty(2, 3, device=DEV), torch.empty(2, 3, 2, device=DEV)
    ctx.token_logps(x, y, logps, row_stats=stats)
    want = lo.token_logps_ref(xn, yn)
    same(logps.cpu().numpy(), want, lp_tolerance(xn, yn, want, 1.0) + U * np.abs(want), "logps")
    coef = torch.ones(2, 3, device=DEV)
    flat = torch.empty(3, 2, 777, device=DEV)
    ctx.token_logps_backward(x, y, stats, coef, flat.transpose(0, 1))
    plain = torch.empty(2, 3, 777, device=DEV)
    ctx.token_logps_backward(x.contiguous(), y, stats, coef, plain)
    assert torch.equal(flat.transpose(0, 1), plain)


def test_two_dimensional_logits_are_one_sequence(ctx):
    x, y, _, _ = make(1, 6, 500, BF)
    out, a, b = torch.empty(4, device=DEV), torch.empty_like(x), torch.empty_like(x)
    ctx.policy_loss(x, y, torch.ones(1, device=DEV), out, grad_logits=a)
    ctx.policy_loss(x[0], y[0], torch.ones(1, device=DEV), out, grad_logits=b[0])
    assert torch.equal(a, b)
    ctx.policy_loss(x[0], y[0], torch.ones(6, device=DEV), out, grad_logits=b[0])
    assert torch.equal(a, b)


def test_refusals_of_the_binding(ctx):
    x, y, _, _ = make(2, 3, 64, BF)
    logps, out = torch.empty(2, 3, device=DEV), torch.empty(4, device=DEV)
    adv = torch.ones(2, device=DEV)
    with pytest.raises(ValueError):
        ctx.token_logps(x.transpose(1, 2), y, logps)           # vocabulary not contiguous
    with pytest.raises(ValueError):
        ctx.token_logps(x[0, 0], y, logps)
    with pytest.raises(ValueError):
        ctx.token_logps(x, y[:, :2].contiguous(), logps)
    with pytest.raises(TypeError):
        ctx.token_logps(x, y.int(), logps)
    with pytest.raises(TypeError):
        ctx.token_logps(x.half(), y, logps)
    with pytest.raises(TypeError):
        ctx.token_logps(x, y, logps.double())
    with pytest.raises(ValueError):
        ctx.token_logps(x, y.cpu(), logps)
    with pytest.raises(ValueError):
        ctx.policy_loss(x, y, adv, out, reduce="mean")
    with pytest.raises(ValueError):
        ctx.policy_loss(x, y, torch.ones(3, device=DEV), out)
    with pytest.raises(ValueError):
        ctx.policy_loss(x, y, adv, out, grad_logits=x.float())
    with pytest.raises(ValueError):
        ctx.preference_loss(x, y, None, torch.empty(3, device=DEV), kind="hinge")
    with pytest.raises(MuonError) as e:
        ctx.policy_loss(x, y, adv, out, kl_coef=0.1)
    assert e.value.status == 1 and "ref_logps" in str(e.value)
    small = Context(DEV, 256)
    with pytest.raises(MuonError) as e:
        small.policy_loss(x, y, adv, out)
    assert e.value.status == 4 and loss_workspace_bytes(2, 3, 64) > 256
    small.close()


def test_other_stream(ctx):
    """Inputs made on one stream, the call on another that waits for it."""
    side = torch.cuda.Stream(DEV)
    x, y, xn, yn = make(1, 64, 4099, BF)
    want = torch.empty(1, 64, device=DEV)
    ctx.token_logps(x, y, want)
    big = torch.randn(2048, 2048, device=DEV)
    for _ in range(8):
        big = big @ big * 1e-3
    x2 = x + 0 * big[0, 0].nan_to_num().to(BF)
    got = torch.empty(1, 64, device=DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    ctx.token_logps(x2, y, got, stream=side)
    torch.cuda.current_stream(DEV).wait_stream(side)
    assert torch.equal(got, want)


@pytest.mark.parametrize("shape", [(2, 8, 50257), (2, 300, 2051)])
def test_recorded_losses_replay(ctx, shape):
    """Both losses in one graph, replayed on new scores and labels with eager
    work between; every replay equals the eager call."""
    batch, seq, vocab = shape
    x, y, _, _ = make(batch, seq, vocab, BF)
    adv, ref = torch.ones(batch, device=DEV), torch.zeros(batch, seq, device=DEV)
    out, out3, grad, grad2 = (torch.empty(4, device=DEV), torch.empty(3, device=DEV), torch.empty_like(x),
                              torch.empty_like(x))

    def both(o, o3, g, g2, stream=None):
        ctx.policy_loss(x, y, adv, o, old_logps=ref, ref_logps=ref, kl_coef=0.01, grad_logits=g, stream=stream)
        ctx.preference_loss(x, y, ref, o3, grad_logits=g2, stream=stream)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.graph(graph, stream=side):
        both(out, out3, grad, grad2, side)
    torch.cuda.current_stream(DEV).wait_stream(side)
    for k in range(4):
        nx, ny, _, _ = make(batch, seq, vocab, BF, seed=20 + k)
        x.copy_(nx)
        y.copy_(ny)
        ref.copy_(torch.randn(batch, seq, device=DEV) - 8)
        graph.replay()
        torch.cuda.synchronize()
        e = [torch.empty_like(v) for v in (out, out3, grad, grad2)]
        both(*e)
        torch.cuda.synchronize()
        for a, b in zip(e, (out, out3, grad, grad2)):
            assert torch.equal(a, b), k


def test_timing_class(ctx):
    x, y, _, _ = make(1, 4, 300, BF)
    c = Context(DEV, 1 << 20)
    c.timing_enable(True, 64)
    c.timing_reset()
    c.token_logps(x, y, torch.empty(1, 4, device=DEV))
    assert c.timing_read()["loss"][1] == 1
    c.close()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_calls_of_one_launch_and_of_several(ctx, dtype):
    """Small calls leave the rest of the work to their last workgroup, which has
    to leave the exchange words empty for the next call: sizes on both sides of
    the limit, in turn, twice; every repeat gives the same bits, and the results
    are the oracle's."""
    shapes = [(2, 512, 300), (2, 513, 300), (2, 1, 151936), (4, 64, 50257), (2, 1, 5), (4, 100, 50257), (16, 64, 77),
              (18, 5, 9001)]
    first = {}
    for turn in range(2):
        for shape in shapes:
            batch, seq, vocab = shape
            x, y, xn, yn = make(batch, seq, vocab, dtype, seed=vocab + seq)
            y[0, 0] = yn[0, 0] = vocab - 1
            y[-1] = yn[-1] = -1  # a whole sequence left out
            ref = torch.full((batch, seq), -9.0, device=DEV)
            lps = [torch.full((batch, seq), 3.0, device=DEV) for _ in range(3)]
            stats, rewards = torch.empty(batch, seq, 2, device=DEV), torch.empty(batch, device=DEV)
            out, out3 = torch.empty(4, device=DEV), torch.empty(3, device=DEV)
            ctx.token_logps(x, y, lps[0], row_stats=stats)
            ctx.preference_loss(x, y, ref, out3, rewards=rewards, logps=lps[1])
            ctx.policy_loss(x, y, torch.ones(batch, device=DEV), out, old_logps=ref, logps=lps[2])
            stats[y < 0] = 0
            got = [v.cpu().numpy() for v in (*lps, stats, rewards, out, out3)]
            if turn:
                for a, b in zip(first[shape], got):
                    assert np.array_equal(a, b), shape
                continue
            first[shape] = got
            lp = lo.token_logps_ref(xn, yn)
            tol = lp_tolerance(xn, yn, lp, 1.0)
            for v in got[:3]:
                same(v, lp, tol + U * np.abs(lp), f"logps {shape}")
            valid = yn >= 0
            score = 0.1 * np.where(valid, lp + 9.0, 0.0).sum(1)
            same(got[4], score, 0.1 * np.where(valid, tol, 0.0).sum(1) + 3 * U * np.abs(score) + 1e-12, f"rewards {shape}")
