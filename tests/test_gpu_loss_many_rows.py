"""Losses over more rows, sequences and pairs than one grid has workgroups for
(needs a gfx950 GPU).

Tolerance of a log-probability, u = 2^-24: its sum is off by at most
u (5 log V + 48) (tests/test_gpu_loss_temperature.py derives it), storing it by
u |lp|; a gradient G ([v = y] - p) by |G| p times that and 10 u |G|."""
import numpy as np
import pytest
import torch

from newton_schulz_amd import Context, loss_workspace_bytes

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
F32 = torch.float32


def log_sum_error(vocab):
    return U * (5 * np.log(vocab) + 48)


def make(batch, vocab):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device=DEV).manual_seed(batch)
    x = torch.empty(batch, 1, vocab, device=DEV).normal_(0.0, 2.0, generator=g)
    y = torch.randint(vocab, (batch, 1), generator=g, device=DEV)
    y[1::5] = -1
    z = torch.log_softmax(x.double(), -1)
    lp = z.gather(-1, y.clamp(min=0).unsqueeze(-1)).squeeze(-1).masked_fill(y < 0, 0.0)
    hot = torch.zeros_like(z).scatter_(-1, y.clamp(min=0).unsqueeze(-1), 1.0)
    return g, x, y, lp, (hot - z.exp()).masked_fill((y < 0).unsqueeze(-1), 0.0)


def within(got, want, tol, what):
    assert bool(((got.double() - want).abs() <= tol).all()), what


def test_sequence_mean_over_more_sequences_than_a_grid():
    batch, vocab = (1 << 22) + 3, 3
    g, x, y, lp, slope = make(batch, vocab)
    adv = torch.empty(batch, device=DEV).normal_(generator=g)
    ctx = Context(DEV, loss_workspace_bytes(batch, 1, vocab, F32))
    out, logps, grad = torch.empty(4, device=DEV), torch.empty(batch, 1, device=DEV), torch.empty_like(x)
    ctx.policy_loss(x, y, adv, out, logps=logps, grad_logits=grad, reduce="sequence", weight=float(batch))
    d = log_sum_error(vocab)
    within(logps, lp, d + U * lp.abs(), "logps")
    G = -adv.double()[:, None, None]
    within(grad, G * slope, G.abs() * (d + 10 * U), "gradient")
    want = (-adv.double() * (y[:, 0] >= 0)).sum().item()
    # binary64 sums of fp32 terms, each with a rounding or two
    assert abs(out[0].item() - want) <= 2 * U * abs(want) + 2 * U * adv.double().abs().sum().item()
    ctx.close()


def test_more_pairs_than_a_grid():
    pairs, vocab, beta = (1 << 22) + 5, 3, 0.5
    g, x, y, lp, slope = make(2 * pairs, vocab)
    ctx = Context(DEV, loss_workspace_bytes(2 * pairs, 1, vocab, F32))
    out, rewards = torch.empty(3, device=DEV), torch.empty(2 * pairs, device=DEV)
    logps, grad = torch.empty(2 * pairs, 1, device=DEV), torch.empty_like(x)
    ctx.preference_loss(x, y, None, out, rewards=rewards, logps=logps, grad_logits=grad, beta=beta, weight=float(pairs))
    d = log_sum_error(vocab)
    within(logps, lp, d + U * lp.abs(), "logps")
    within(rewards, beta * lp[:, 0], beta * d + U * lp[:, 0].abs(), "rewards")
    h = beta * (lp[:pairs, 0] - lp[pairs:, 0])
    loss = torch.nn.functional.softplus(-h, threshold=1e9).mean().item()
    # out[0] = pairs * the mean; a pair's loss moves by at most beta 2 d
    assert abs(out[0].item() / pairs - loss) <= 2 * beta * d + 2 * U * loss
    slopes = -beta * torch.sigmoid(-h)
    G = torch.cat([slopes, -slopes])[:, None, None]
    # the slope itself by beta^2 / 4 2 d
    within(grad, G * slope, G.abs() * (d + 10 * U) + 0.5 * beta * beta * d, "gradient")
    ctx.close()


def test_more_rows_of_several_slices_than_a_grid_has_waves():
    """2^26 + 9 rows, all the same one in memory, nearly all of them left out."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rows, vocab = (1 << 26) + 9, 20488
    x = torch.randn(1, 1, vocab, device=DEV).bfloat16()
    y = torch.full((1, rows), -1, dtype=torch.int64, device=DEV)
    at = torch.tensor([0, 1, 3, 4_000_001, (1 << 26) - 1, 1 << 26, (1 << 26) + 5, rows - 1], device=DEV)
    y[0, at] = torch.arange(8, device=DEV) * 2900
    logps = torch.full((1, rows), 5.0, device=DEV)
    ctx = Context(DEV, loss_workspace_bytes(1, rows, vocab))
    ctx.token_logps(x.expand(1, rows, vocab), y, logps)
    want = torch.log_softmax(x.double(), -1)[0, 0, y[0, at]]
    within(logps[0, at], want, log_sum_error(vocab) + U * want.abs(), "logps")
    logps[0, at] = 0.0
    assert not logps.any()
    ctx.close()
