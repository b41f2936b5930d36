"""CPU oracle for the losses in front of the optimizer step and for gradient
clipping: numpy, binary64, straight from the definitions.

TEST INFRASTRUCTURE ONLY, as muon_oracle.py is: the product path shares no
code with it.

With z = x / T, label y of a row, lse = log sum_v exp z_v:
  * lp = z_y - lse; d lp / d x_v = ([v = y] - exp(z_v - lse)) / T.  A negative
    label leaves the token out (lp 0, gradient 0), one >= V gives NaN.
  * policy: r = exp(lp - old), pg = max(-A r, -A clip(r, 1 - lo, 1 + hi)),
    e = ref - lp, kl = exp e - 1 - e, loss = sum_t w_t (pg + c kl); w = 1 / N,
    1 / (batch n_b), or 1.
  * preference: s_i = sum (or mean) of lp - ref, m = s_i - s_{P+i}, sigmoid
    -(1 - eps) log sigma(beta m) - eps log sigma(-beta m), ipo
    (m - 1 / (2 beta))^2, mean over the P pairs.
  * clipping: S = sum g^2, coefficient min(1, max_norm / (sqrt S + eps)).

The gradients are written out here and pinned by central differences of the
losses (tests/test_oracle_losses.py).
"""
from __future__ import annotations

import math

import numpy as np


def token_logps_ref(x, y, temperature=1.0):
    """lp of every row of x [..., V] (float64) for labels y [...]."""
    x = np.asarray(x, np.float64)
    z = x.reshape(-1, x.shape[-1]) / temperature
    lab = np.asarray(y).reshape(-1)
    out = np.zeros(len(lab))
    with np.errstate(all="ignore"):
        for i, (row, k) in enumerate(zip(z, lab)):
            if k < 0:
                continue
            if k >= len(row):
                out[i] = np.nan
                continue
            top = row.max()
            out[i] = row[k] - top - np.log(np.exp(row - top).sum())
    return out.reshape(np.shape(y))


def softmax_ref(x, temperature=1.0):
    with np.errstate(all="ignore"):
        z = np.asarray(x, np.float64) / temperature
        e = np.exp(z - z.max(-1, keepdims=True))
        return e / e.sum(-1, keepdims=True)


def logits_grad_ref(x, y, g, temperature=1.0):
    """Gradient of sum_t g_t lp_t in x."""
    x = np.asarray(x, np.float64)
    p = softmax_ref(x, temperature).reshape(-1, x.shape[-1])
    lab, gg = np.asarray(y).reshape(-1), np.asarray(g, np.float64).reshape(-1)
    out = np.zeros_like(p)
    with np.errstate(all="ignore"):
        for i, k in enumerate(lab):
            if k < 0:
                continue
            out[i] = -gg[i] / temperature * p[i]
            if k < p.shape[1]:
                out[i, k] += gg[i] / temperature
            else:
                out[i] = np.nan
    return out.reshape(x.shape)


def policy_weights(y, reduce):
    valid = np.asarray(y) >= 0
    n = valid.sum(1, keepdims=True)
    if reduce == "token":
        w = np.full(valid.shape, 1.0 / max(1, int(n.sum())))
    elif reduce == "sequence":
        w = np.broadcast_to(1.0 / (np.maximum(n, 1) * valid.shape[0]), valid.shape)
    else:
        w = np.ones(valid.shape)
    return np.where(valid, w, 0.0)


def policy_ref(lp, y, adv, old=None, ref=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0, reduce="token",
               weight=1.0):
    """({loss, pg, kl, clipped}, gradient in lp) of the policy loss."""
    valid = np.asarray(y) >= 0
    lp = np.asarray(lp, np.float64)
    a = np.asarray(adv, np.float64)
    a = np.broadcast_to(a[:, None] if a.ndim == 1 else a, lp.shape)
    w = policy_weights(y, reduce)
    with np.errstate(all="ignore"):
        r = np.exp(lp - np.asarray(old, np.float64)) if old is not None else np.where(np.isnan(lp), lp, 1.0)
        free, held = -a * r, -a * np.clip(r, 1.0 - clip_low, 1.0 + clip_high)
        pg = np.maximum(free, held)
        g = np.where(held > free, 0.0, free)
        kl = np.zeros_like(lp)
        if ref is not None:
            e = np.asarray(ref, np.float64) - lp
            kl = np.expm1(e) - e
            if kl_coef:
                g = g - kl_coef * np.expm1(e)
        total = [np.where(valid, w * v, 0.0).sum() for v in (pg, kl, (held > free).astype(float))]
        g = np.where(valid, weight * w * g, 0.0)
    loss = total[0] + (kl_coef * total[1] if kl_coef else 0.0)
    return np.array([weight * loss, *total]), g


def preference_ref(lp, y, ref=None, kind="sigmoid", beta=0.1, label_smoothing=0.0, average=False, weight=1.0):
    """({loss, mean margin, share right}, rewards, gradient in lp)."""
    valid = np.asarray(y) >= 0
    lp = np.asarray(lp, np.float64)
    pairs = lp.shape[0] // 2
    n = np.maximum(valid.sum(1, keepdims=True), 1) if average else np.ones((lp.shape[0], 1))
    part = np.where(valid, 1.0 / n, 0.0)
    score = np.where(valid, part * (lp - (np.asarray(ref, np.float64) if ref is not None else 0.0)), 0.0).sum(1)
    m = score[:pairs] - score[pairs:]
    h = beta * m
    if kind == "sigmoid":
        loss = (1 - label_smoothing) * np.logaddexp(0, -h)
        if label_smoothing:
            loss = loss + label_smoothing * np.logaddexp(0, h)
        sig = np.exp(-np.logaddexp(0, -h))
        d = beta * (label_smoothing * sig - (1 - label_smoothing) * np.exp(-np.logaddexp(0, h)))
    else:
        loss, d = (m - 0.5 / beta) ** 2, 2 * (m - 0.5 / beta)
    d = weight * d / max(1, pairs)
    g = np.concatenate([d, -d])[:, None] * part if pairs else np.zeros_like(lp)
    k = max(1, pairs)
    return np.array([weight * loss.sum() / k, h.sum() / k, (m > 0).sum() / k]), beta * score, g


def grad_norm_ref(tensors, max_norm, eps=1e-6):
    """{S, sqrt S, coefficient}; S exactly rounded."""
    s = math.fsum(float(v) for t in tensors for v in np.square(np.asarray(t, np.float64)).reshape(-1))
    size = math.sqrt(s)
    return s, size, min(1.0, max_norm / (size + eps)) if size + eps > 0 else 1.0
