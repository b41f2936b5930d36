"""Preference pairs with an answer that the policy gives no probability at all
(needs a gfx950 GPU)."""
import math

import pytest
import torch

from newton_schulz_amd import Context

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF = float("inf")


@pytest.mark.parametrize("pairs", [1, 20])
@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_impossible_answers(pairs, smoothing):
    """A masked token in the rejected answer makes the margin infinite: the loss
    of the pair is 0 and so is its gradient; with smoothing, or in the chosen
    answer, the loss is infinite and the gradient finite."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    vocab, seq, beta = 37, 3, 0.5
    g = torch.Generator(device=DEV).manual_seed(pairs)
    x = torch.empty(2 * pairs, seq, vocab, device=DEV).normal_(generator=g)
    y = torch.zeros(2 * pairs, seq, dtype=torch.int64, device=DEV)
    ctx = Context(DEV, 1 << 20)
    out, rewards = torch.empty(3, device=DEV), torch.empty(2 * pairs, device=DEV)
    finite, grad = torch.empty(3, device=DEV), torch.empty_like(x)
    rest = x.clone()
    rest[0, :, 1:], rest[pairs, :, 1:] = -INF, -INF  # a first pair of lp 0 and 0: log 2
    ctx.preference_loss(rest, y, None, finite, beta=beta, label_smoothing=smoothing)
    masked = x.clone()
    masked[pairs, 1, 0] = -INF  # the first pair's rejected answer
    ctx.preference_loss(masked, y, None, out, rewards=rewards, grad_logits=grad, beta=beta, label_smoothing=smoothing)
    assert rewards[pairs] == -INF and out[1] == INF and rewards.isfinite().sum() == 2 * pairs - 1
    if smoothing:
        assert out[0] == INF
        # slope beta * smoothing / pairs of the margin: a rejected token's gradient -that ([v = y] - p)
        k = beta * smoothing / pairs
        want = torch.softmax(masked[pairs].double(), -1) * k
        want[:, 0] -= k
        # fp32 p and factor, a few roundings each
        assert bool(((grad[pairs].double() - want).abs() <= 64 * 2.0 ** -24 * k).all())
    else:
        # the other pairs' losses alone: each fp32 value has one rounding
        want = finite[0].item() - math.log(2) / pairs
        assert out[0].item() == pytest.approx(want, abs=4 * 2.0 ** -24)
        assert not grad[0].any() and not grad[pairs].any()
    assert grad.isfinite().all()
    masked = x.clone()
    masked[0, 2, 0] = -INF  # the first pair's chosen answer
    ctx.preference_loss(masked, y, None, out, rewards=rewards, grad_logits=grad, beta=beta, label_smoothing=smoothing)
    assert out[0] == INF and out[1] == -INF and rewards[0] == -INF and grad.isfinite().all()
    ctx.close()
