"""Losses at temperatures far from 1 against the binary64 oracle (needs a gfx950
GPU).

k = log2 e / T is held as fp32 and a rest.  From T = 8.6e-8 down (k above 2^24) the
rest can exceed 1 in magnitude, and the product of the lowest number, which the
running maximum starts from, with it leaves fp32.

Tolerances, u = 2^-24, z = x / T, M the row's maximum: an exponential's argument is off by
at most 5 u |z - M| (the difference, the product, and k up or down by 2 u and its
mean), the exponential by 2 u, three additions of a piece by 3 u, and every
raise of the maximum (a piece or an edge each at most: 12 in rows of one slice)
or join (2) scales by a factor off by 3 u beside its argument.  Averaged with
the softmax, M - z is at most log V.  So log S is off by at most
u (5 log V + 2 + 3 + 42 + 1), lp by that and u |lp| of storing it.  A gradient's p
is off by p (that + u (4 |z - M| + 8)); storing rounds by half a step; p below 2^-126 may be 0."""
import numpy as np
import pytest
import torch

from newton_schulz_amd import Context
from oracle import loss_oracle as lo

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
LOG2E = 1.4426950408889634


def rest(t):
    return LOG2E / t - float(np.float32(LOG2E / t))


# rests of either sign, above and below 1 in magnitude
TEMPERATURES = [1e29, 1e6, 1e-4, 5e-8, 3e-8, 1e-8, 7e-9, 3e-9, 7e-10, 1e-10, 7e-12, 1e-12, 1e-20, 3e-20, 1e-28, 2e-30]


def test_rests_of_either_sign():
    small = [rest(t) for t in TEMPERATURES if t < 8e-8]
    assert sum(r < -1 for r in small) >= 2 and sum(r > 1 for r in small) >= 2


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t", TEMPERATURES)
@pytest.mark.parametrize("vocab", [777, 20011])
def test_losses_at_any_temperature(t, vocab, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(vocab)
    # scores of the size of the temperature: an ordinary softmax; the last row of
    # ordinary size, whose softmax is (nearly) one score, if T is small
    x = torch.randn(1, 9, vocab, generator=g, dtype=torch.float64) * 3
    x[0, :8] *= t
    x = x.clamp(-1e30, 1e30).to(dtype)
    x[0, 3, ::5] = -float("inf")
    y = torch.randint(vocab, (1, 9), generator=g)
    y[0, 3], y[0, 4], y[0, 8] = 1, -1, x[0, 8].double().argmax()
    xn, yn = x.double().numpy(), y.numpy()
    want = lo.token_logps_ref(xn, yn, t)
    assert np.isfinite(want).all()
    log_s = U * (5 * np.log(vocab) + 48)
    tol = np.where(yn >= 0, log_s + 2 * U * np.abs(want), 0.0)
    ctx = Context(DEV, 1 << 20)
    xd, yd = x.to(DEV), y.to(DEV)
    logps, stats = torch.empty(1, 9, device=DEV), torch.empty(1, 9, 2, device=DEV)
    ctx.token_logps(xd, yd, logps, row_stats=stats, temperature=t)
    off = np.abs(logps.double().cpu().numpy() - want)
    assert (off <= tol).all(), (off - tol).max()

    # the gradient, of a weight that keeps weight / T in range
    weight = min(1.0, 1e20 * t)
    p = lo.softmax_ref(xn, t)
    z = xn / t
    with np.errstate(invalid="ignore"):
        far = np.where(np.isfinite(z), z.max(-1, keepdims=True) - z, 0.0)
    w32 = float(np.float32(weight))
    gw = lo.logits_grad_ref(xn, yn, np.full((1, 9), w32), t)
    G = w32 / t
    own = np.arange(vocab) == yn[..., None]
    g_tol = G * (np.where(far < 87, p * (log_s + U * (4 * far + 8)), p) + own * (tol + 8 * U * np.abs(np.expm1(want)))[..., None])
    g_tol = g_tol * 1.01 + np.abs(gw) * torch.finfo(dtype).eps / 2 + 2.0 ** -126
    coef, grad = torch.full((1, 9), weight, device=DEV), torch.empty_like(xd)
    ctx.token_logps_backward(xd, yd, stats, coef, grad, temperature=t)
    off = np.abs(grad.double().cpu().numpy() - gw)
    assert (off <= g_tol).all(), (off - g_tol).max()

    # the policy loss at its own policy: the same gradient, times its factor
    out, g2 = torch.empty(4, device=DEV), torch.empty_like(xd)
    ctx.policy_loss(xd, yd, torch.full((1,), -1.0, device=DEV), out, logps=logps, grad_logits=g2, reduce="sum",
                    weight=weight, temperature=t)
    assert (np.abs(logps.double().cpu().numpy() - want) <= tol).all()
    off = np.abs(g2.double().cpu().numpy() - gw)
    assert (off <= g_tol).all(), (off - g_tol).max()
    assert out[0].item() == pytest.approx(weight * 8, rel=4 * U)

    # the preference loss without a reference
    x2, y2 = xd.expand(2, 9, vocab).contiguous(), torch.stack([yd[0], torch.full_like(yd[0], -1)])
    out3, rewards = torch.empty(3, device=DEV), torch.empty(2, device=DEV)
    ctx.preference_loss(x2, y2, None, out3, rewards=rewards, beta=0.25, temperature=t)
    score = want.sum()
    assert abs(rewards[0].item() - 0.25 * score) <= 0.25 * tol.sum() + U * abs(0.25 * score) and rewards[1] == 0
    ctx.close()
