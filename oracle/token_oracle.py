"""Plain fp64 CPU oracle of the token log-probabilities and gradient clipping.

TEST INFRASTRUCTURE ONLY, written from the definitions (include/kd.h,
kd_logprob_* and kd_clip_grad_norm); it shares no code with the CUDA library.
Rows of materialised logits; a = z / T, p = softmax(a).  Pinned by closed
forms, finite differences and brute force in tests/test_token_oracle.py.
"""
from __future__ import annotations

import math

import numpy as np

from .kd_oracle import as_f64


def _row(z, t):
    """(log p, p, entropy) of one row of finite or -inf logits."""
    a = z / t
    m = a.max()
    e = np.exp(a - m)
    lp = a - m - math.log(e.sum())
    p = np.exp(lp)
    return lp, p, -float(np.sum(p[p > 0] * lp[p > 0]))


def top_ids(z, k):
    """Ids of the k largest: a NaN above every number, equal values by id."""
    key = [(0 if math.isnan(x) else 1, -x if not math.isnan(x) else 0.0, i)
           for i, x in enumerate(z.tolist())]
    return [i for _, _, i in sorted(key)[:k]]


def forward(z, tokens, *, temperature=1.0, topk=0, ignore_index=-100):
    z = as_f64(z)
    n, v = z.shape
    nan, inf = math.nan, math.inf
    out = {"logprob": np.zeros(n), "entropy": np.zeros(n),
           "topk_idx": np.tile(np.arange(topk), (n, 1)), "topk_logprob": np.full((n, topk), -inf)}
    for r in range(n):
        y = None if tokens is None else int(tokens[r])
        if y is not None and y == ignore_index:
            continue
        if np.isnan(z[r]).any() or (z[r] == inf).any():
            lp, ent = np.full(v, nan), nan
        elif (z[r] == -inf).all():
            lp, ent = np.full(v, -inf), 0.0
        else:
            with np.errstate(divide="ignore"):
                lp, _, ent = _row(z[r], temperature)
        out["entropy"][r] = ent
        if y is not None:
            out["logprob"][r] = lp[y] if 0 <= y < v else nan
        ids = top_ids(z[r], topk)
        out["topk_idx"][r] = ids
        out["topk_logprob"][r] = lp[ids]
    return out


def grad_logits(z, tokens, d_logprob, d_entropy, *, temperature=1.0, ignore_index=-100):
    """d/dz of sum_n d_logprob[n] logprob[n] + d_entropy[n] entropy[n]."""
    z = as_f64(z)
    g = np.zeros_like(z)
    for r in range(len(z)):
        y = None if tokens is None else int(tokens[r])
        if (y is not None and y == ignore_index) or (z[r] == -math.inf).all():
            continue
        lp, p, ent = _row(z[r], temperature)
        bad = y is not None and not 0 <= y < z.shape[1]
        gl = 0.0 if d_logprob is None or y is None or bad else float(d_logprob[r])
        gh = 0.0 if d_entropy is None else float(d_entropy[r])
        on = p > 0
        g[r, on] = -p[on] * (gl + gh * (lp[on] + ent))
        if gl:
            g[r, y] += gl
    return g / temperature


def clip(grads, max_norm):
    """(norm, clipped gradients)."""
    gs = [as_f64(g) for g in grads]
    big = max([float(np.abs(g).max()) for g in gs if g.size] + [0.0]) or 1.0
    norm = math.sqrt(math.fsum(float(np.sum((g / big) ** 2)) for g in gs)) * big
    return norm, [g * (max_norm / norm if norm > max_norm else 1.0) for g in gs]
