"""How far log-probabilities over large vocabularies are off: every one of them,
their mean, and a sequence's sum (needs a gfx950 GPU but for the first test).

u = 2^-24, z = x / T, M a row's maximum, E = sum p (M - z).

One row.  An exponential's argument is off by at most 5 u |z - M| (difference,
product, and k = log2 e / T, which is one of the two fp32 numbers next to it and has
2 u; factors between maxima take 2 u of the way they span), it itself by 2 u, three
additions in fp32 by 3 u; beyond these sums are binary64.  A score passes at most
11 raises of its wave's maximum and 2 joins, 3 u each, and S - 1 is stored once or
twice, u each.  Averaged with p, log S is off by at most u (5 E + 46).

The mean of many rows.  Roundings have no preferred direction; what has one is k.
It is rounded up in n of the 8 (fp32: 4) places of 16 bytes so that its mean is
right, but n is whole: half a place of 8 is 1/16 of a step of k, at most u / 8 of
it (fp32: u / 4).  So the mean of log S is off by E u / 8 (E u / 4) and what the
roundings leave: of the exponential instruction u / 4 is granted, of the rest
five standard deviations of at most u a row with 20 rows that differ (bf16 maxima
lie on few values): 5 u / sqrt(20)."""
import numpy as np
import pytest
import torch

from newton_schulz_amd import Context, loss_workspace_bytes

DEV = "cuda:0"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
LOG2E = 1.4426950408889634
# k half a step and 1/16 of a step above an fp32 number next to 1, and ordinary ones
TEMPERATURES = [LOG2E / (1 + 2.0 ** -24), LOG2E / (1 + 2.0 ** -27), 0.83, 1.0]


def row_tolerance(e):
    return U * (5 * e + 46)


def mean_tolerance(e, dtype):
    return U * (e / (8 if dtype == BF else 4) + 0.25 + 5 / 20 ** 0.5)


def exact(x, t):
    """(log S around the maximum, E) of rows, binary64."""
    z = x.double() / t
    d = z.amax(-1, keepdim=True) - z
    w = (-d).exp()
    s = w.sum(-1)
    return s.log(), (w * d).sum(-1) / s


def test_the_mean_finds_a_rounded_temperature():
    """With k rounded to fp32 everywhere, and no other error at all, the mean is
    far outside at the first temperature."""
    t = TEMPERATURES[0]
    x = (torch.randn(24, 50257, generator=torch.Generator().manual_seed(0)) * (2 * t)).to(BF)
    want, e = exact(x, t)
    d = x.double() - x.double().amax(-1, keepdim=True)
    got = torch.exp2(d * float(np.float32(LOG2E / t))).sum(-1).log()
    for dtype in (BF, F32):
        assert (got - want).mean().abs() > 1.5 * mean_tolerance(e.mean().item(), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [50257, 151936])
@pytest.mark.parametrize("t", TEMPERATURES)
def test_rows_mean_and_sum(t, vocab, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    seq = 512
    g = torch.Generator(device=DEV).manual_seed(vocab)
    x = torch.empty(2, seq, vocab, dtype=dtype, device=DEV).normal_(0.0, 2.0 * t, generator=g)
    y = torch.randint(vocab, (2, seq), generator=g, device=DEV)
    parts = [exact(r, t) for r in x.view(-1, vocab).split(64)]
    log_s, e = (torch.cat(v).view(2, seq) for v in zip(*parts))
    zy = x.gather(-1, y.unsqueeze(-1)).squeeze(-1).double() / t
    lp = zy - x.amax(-1).double() / t - log_s

    ctx = Context(DEV, loss_workspace_bytes(2, seq, vocab, dtype))
    logps, stats = torch.empty(2, seq, device=DEV), torch.empty(2, seq, 2, device=DEV)
    ctx.token_logps(x, y, logps, row_stats=stats, temperature=t)
    off = torch.log1p(stats[..., 1].double()) - log_s
    assert bool((off.abs() <= row_tolerance(e)).all()), (off.abs().max() / U).item()
    assert bool(((logps.double() - lp).abs() <= row_tolerance(e) + U * lp.abs()).all())
    mean = off.mean().item()
    print(f"mean {mean / U:+.3f} u, rows {off.std().item() / U:.3f} u, worst {off.abs().max().item() / U:.2f} u", flush=True)
    assert abs(mean) <= mean_tolerance(e.mean().item(), dtype), mean / U

    # a sequence's sum, against a reference that leaves little of it to round
    ref, out, rewards = lp.float(), torch.empty(3, device=DEV), torch.empty(2, device=DEV)
    ctx.preference_loss(x, y, ref, out, rewards=rewards, beta=1.0, temperature=t)
    want = (lp - ref.double()).sum(-1)
    tol = seq * mean_tolerance(e.mean(-1), dtype) + U * want.abs() + 1e-9
    assert bool(((rewards.double() - want).abs() <= tol).all()), ((rewards.double() - want) / seq / U).tolist()
    ctx.close()
