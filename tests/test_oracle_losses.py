"""The loss oracle against facts other than itself: central differences,
closed forms, scipy's logsumexp.  No GPU."""
import numpy as np
import pytest
from scipy.special import logsumexp

from oracle import loss_oracle as lo


def test_logps_match_logsumexp_and_sum_to_one(rng):
    x = rng.normal(0, 4, (6, 50))
    for t in (0.5, 1.0, 2.0):
        every = np.stack([lo.token_logps_ref(x, np.full(6, k), t) for k in range(50)], 1)
        want = x / t - logsumexp(x / t, axis=1, keepdims=True)
        assert np.abs(every - want).max() < 1e-13
        assert np.abs(np.exp(every).sum(1) - 1).max() < 1e-13


def test_logps_of_special_rows():
    inf = np.inf
    x = np.array([[-inf, 1.0, 1.0], [-inf, -inf, -inf], [inf, 0.0, 0.0], [np.nan, 0.0, 0.0], [0.0, 0.0, 0.0]])
    lp = lo.token_logps_ref(x, np.array([1, 0, 1, 1, 3]))
    assert lp[0] == pytest.approx(-np.log(2)) and np.isnan(lp[1:]).all()
    assert lo.token_logps_ref(x[:1], np.array([0]))[0] == -inf
    assert (lo.token_logps_ref(x, np.full(5, -100)) == 0).all()


def _difference(f, v, h=1e-6):
    g = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        up, down = v.copy(), v.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


def test_logits_gradient_is_the_difference_quotient(rng):
    x, y, c = rng.normal(0, 2, (2, 3, 7)), rng.integers(0, 7, (2, 3)), rng.normal(size=(2, 3))
    y[0, 1] = -1
    f = lambda v: float((c * lo.token_logps_ref(v, y, 0.7)).sum())
    assert np.abs(_difference(f, x) - lo.logits_grad_ref(x, y, c, 0.7)).max() < 1e-8


@pytest.mark.parametrize("reduce", ["token", "sequence", "sum"])
@pytest.mark.parametrize("per_token", [False, True])
def test_policy_gradient_is_the_difference_quotient(rng, reduce, per_token):
    lp = -rng.uniform(0.1, 5, (3, 6))
    y = rng.integers(0, 9, (3, 6))
    y[0, :2] = -100
    y[2] = -100
    old, ref = lp + rng.normal(0, 0.4, lp.shape), lp + rng.normal(0, 0.4, lp.shape)
    adv = rng.normal(size=lp.shape if per_token else 3)
    # one token that the clip holds: ratio e, positive advantage
    y[1, 0], old[1, 0] = 3, lp[1, 0] - 1.0
    adv[1] = np.abs(adv[1])
    kw = dict(old=old, ref=ref, clip_low=0.2, clip_high=0.3, kl_coef=0.1, reduce=reduce, weight=0.5)
    out, g = lo.policy_ref(lp, y, adv, **kw)
    assert np.abs(_difference(lambda v: lo.policy_ref(v, y, adv, **kw)[0][0], lp) - g).max() < 1e-7
    assert out[3] > 0 and (g[2] == 0).all() and (g[0, :2] == 0).all()
    # hand-written: every term one at a time
    n = (y >= 0).sum()
    want = 0.0
    for b in range(3):
        for t in range(6):
            if y[b, t] < 0:
                continue
            w = {"token": 1 / n, "sequence": 1 / (3 * max(1, (y[b] >= 0).sum())), "sum": 1.0}[reduce]
            a = adv[b, t] if per_token else adv[b]
            r = np.exp(lp[b, t] - old[b, t])
            want += w * (-min(a * r, a * min(max(r, 0.8), 1.3))
                         + 0.1 * (np.exp(ref[b, t] - lp[b, t]) - 1 - ref[b, t] + lp[b, t]))
    assert out[0] == pytest.approx(0.5 * want, rel=1e-12)


def test_policy_of_its_own_policy_is_the_plain_gradient(rng):
    lp, y, adv = -rng.uniform(0.1, 5, (2, 4)), np.zeros((2, 4), int), rng.normal(size=2)
    out, g = lo.policy_ref(lp, y, adv)
    assert out[0] == pytest.approx(-adv.mean()) and np.allclose(g, -adv[:, None] / 8)


@pytest.mark.parametrize("kind,eps,average", [("sigmoid", 0.0, False), ("sigmoid", 0.1, True), ("ipo", 0.0, True),
                                              ("ipo", 0.0, False)])
def test_preference_gradient_is_the_difference_quotient(rng, kind, eps, average):
    lp = -rng.uniform(0.1, 5, (4, 5))
    y = rng.integers(0, 9, (4, 5))
    y[0, 3:] = -1
    y[3] = -1
    ref = lp + rng.normal(0, 0.5, lp.shape)
    kw = dict(ref=ref, kind=kind, beta=0.3, label_smoothing=eps, average=average, weight=2.0)
    out, rewards, g = lo.preference_ref(lp, y, **kw)
    assert np.abs(_difference(lambda v: lo.preference_ref(v, y, **kw)[0][0], lp) - g).max() < 1e-7
    assert rewards[3] == 0 and (g[y < 0] == 0).all()


def test_preference_closed_forms():
    lp = np.array([[-1.0], [-1.0]])
    out, rewards, g = lo.preference_ref(lp, np.zeros((2, 1), int), beta=0.5)
    assert out[0] == pytest.approx(np.log(2)) and out[2] == 0
    assert np.allclose(g[:, 0], [-0.25, 0.25]) and np.allclose(rewards, -0.5)


def test_grad_norm_pins(rng):
    s, size, c = lo.grad_norm_ref([np.full(9, 2.0), np.full(7, -1.0)], 1.0, 0.0)
    assert (s, size, c) == (43.0, np.sqrt(43.0), 1 / np.sqrt(43.0))
    assert lo.grad_norm_ref([np.full(4, 0.1)], 1.0)[2] == 1.0
