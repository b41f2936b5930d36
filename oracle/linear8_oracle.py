"""CPU oracle for 8-bit linear layers and draft verification: numpy, straight
from the definitions.

TEST INFRASTRUCTURE ONLY, as muon_oracle.py is: the product path shares no
code with it.

  * rows in 8 bits: scale = fp32(max |x| / 127), q the integer nearest to the
    exact x / scale, ties to even (fractions of integers decide: nothing is
    rounded on the way), 0 for rows of zeros, scale NaN and q 0 for rows with
    anything not finite.
  * product: fp32(sum of integers) * fp32(sa * sb), rounded to fp32.
  * gradients: grad_x = grad_y w, grad_w = grad_y^T x with w, x = scale * q.
  * verification: place i keeps its drafted token x while u_i q_i(x) < p_i(x);
    the first that does not takes the lowest v whose weights max(p - q, 0) up
    to it exceed u_K times their sum.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def quantize_ref(x):
    """(q int8, scale float32) of the rows of x (float32 values)."""
    x = np.asarray(x, np.float32)
    q, scale = np.zeros(x.shape, np.int8), np.zeros(len(x), np.float32)
    for r, row in enumerate(x):
        if not np.isfinite(row).all():
            scale[r] = np.nan
            continue
        s = min(np.float32(np.abs(row).max()) / np.float32(127.0), np.float32(float.fromhex("0x1.020406p+121")))
        scale[r] = s
        if s == 0:
            continue
        d = row.astype(np.float64) / np.float64(s)  # right to 2^-53
        n = np.rint(d)
        # next to a half the exact quotient decides
        for c in np.nonzero(np.abs(np.abs(d - np.floor(d)) - 0.5) < 1e-9)[0]:
            n[c] = round(Fraction(float(row[c])) / Fraction(float(s)))  # (ties to even)
        q[r] = np.clip(n, -127, 127).astype(np.int8)
    return q, scale


def matmul8_ref(qa, sa, qb, sb):
    """float32 product of 8-bit rows, as it is rounded."""
    total = qa.astype(np.int64) @ qb.astype(np.int64).T
    with np.errstate(all="ignore"):
        return total.astype(np.float32) * (sa[:, None] * sb[None, :])


def values_ref(q, scale):
    with np.errstate(all="ignore"):
        return q.astype(np.float64) * scale.astype(np.float64)[:, None]


def softmax_row(x, t):
    """float64 probabilities, or None where the row has no distribution."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all():
        return None
    e = np.exp((x - x.max()) / t)
    return e / e.sum()


def verify_ref(logits, draft, draft_logits, uniforms, temperature):
    """tokens, accepted, logps of each sequence; logits [B, K + 1, V] float64."""
    B, K1, V = logits.shape
    tokens = np.full((B, K1), -1, np.int64)
    accepted = np.zeros(B, np.int64)
    logps = np.zeros((B, K1))
    t = temperature or 1.0
    for b in range(B):
        i = 0
        while True:
            p = softmax_row(logits[b, i], t)
            y = int(draft[b, i]) if i < K1 - 1 else -1
            if p is None:
                logps[b, i] = np.nan
                break
            if temperature == 0:
                take = int(np.argmax(logits[b, i]))
                keep = y == take
            else:
                q = None
                if y >= 0:
                    if draft_logits is not None:
                        q = softmax_row(draft_logits[b, i], t)
                    else:
                        q = np.zeros(V)
                        if y < V:
                            q[y] = 1.0
                keep = 0 <= y < V and q is not None and float(uniforms[b, i]) * q[y] < p[y]
                if not keep:
                    w = p if q is None else np.maximum(p - q, 0.0)
                    if not w.sum() > 0:
                        w = p
                    edges = np.cumsum(w)
                    inside = np.nonzero((edges > float(uniforms[b, -1]) * edges[-1]) & (w > 0))[0]
                    take = int(inside[0]) if len(inside) else int(np.nonzero(w > 0)[0][-1])
            tokens[b, i] = y if keep else take
            with np.errstate(all="ignore"):
                x = np.asarray(logits[b, i], np.float64)
                top = x.max()
                logps[b, i] = (x[tokens[b, i]] - top) / t - np.log(np.exp((x - top) / t).sum())
            if not keep:
                break
            i += 1
        accepted[b] = i
    return tokens, accepted, logps
