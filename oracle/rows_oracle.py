"""Plain fp64 CPU oracle of draft verification, the embedding and its
gradient, and the root-mean-square norm.

TEST INFRASTRUCTURE ONLY, written from the definitions (include/kd.h,
kd_verify_drafts, kd_embed_*, kd_rmsnorm_*), row by row; it shares no code with
the CUDA library.  Pinned in tests/test_rows_oracle.py.
"""
from __future__ import annotations

import numpy as np

from .kd_oracle import as_f64


def _softmax(z, t):
    """Probabilities of one row, or None where it has no distribution."""
    if np.isnan(z).any() or (z == np.inf).any() or (z == -np.inf).all():
        return None
    a = (z - z.max()) / t
    e = np.exp(a)
    return e / e.sum()


def race(weight, noise):
    """(first arrival, how far ahead of the second it is: the ratio of their times)."""
    w = np.where((noise >= 2.0 ** -60) & (noise <= 2.0 ** 60), weight, 0.0)
    with np.errstate(divide="ignore"):
        time = np.where(w > 0, noise / w, np.inf)
    first = int(np.argmin(time))
    if not np.isfinite(time[first]):
        return None, np.inf
    rest = np.delete(time, first)
    return first, (rest.min() / time[first] if rest.size else np.inf)


def verify(target, draft, drafts, lengths, uniform, noise, *, t_target=1.0, t_draft=1.0,
           ignore_index=-100):
    """dict(tokens, accepted, logprob, bad_label, nonfinite, margin); ``margin``
    [B]: the smallest |u q / p - 1| of the decisions taken and ratio - 1 of the
    race (how far each sequence is from a border)."""
    target = as_f64(target)
    draft = None if draft is None else as_f64(draft)
    drafts, noise = np.asarray(drafts), None if noise is None else as_f64(noise)
    uniform = None if uniform is None else as_f64(uniform)
    b, rows, v = target.shape
    k = rows - 1
    out = {"tokens": np.full((b, rows), ignore_index, np.int64), "accepted": np.zeros(b, np.int32),
           "logprob": np.zeros((b, rows)), "bad_label": False, "nonfinite": False,
           "margin": np.full(b, np.inf)}
    t = t_target or 1.0
    for s in range(b):
        length = k if lengths is None else int(lengths[s])
        if length > k:
            out["bad_label"], length = True, k
        if length < 0:
            continue
        n, weight, live = 0, None, True
        while True:
            z = target[s, n]
            p = _softmax(z, t)
            live = p is not None
            weight = p
            if n == length:
                out["nonfinite"] |= not live
                break
            x = int(drafts[s, n])
            known = 0 <= x < v
            out["bad_label"] |= not known
            if t_target == 0.0:
                if not live:
                    out["nonfinite"] = True
                    break
                if not known or int(np.argmax(z)) != x:
                    break
            else:
                q = None
                if draft is None:
                    q = np.zeros(v)
                    if known:
                        q[x] = 1.0
                else:
                    q = _softmax(draft[s, n], t_draft)
                if not live or q is None:
                    out["nonfinite"] = True
                    break
                ok = False
                if known:
                    lhs = float(uniform[s, n]) * q[x]
                    ok = lhs < p[x]
                    far = abs(lhs / p[x] - 1.0) if p[x] > 0 else np.inf
                    out["margin"][s] = min(out["margin"][s], far)
                if not ok:
                    rest = np.maximum(p - q, 0.0)
                    weight = rest if (rest > 0).any() else p
                    break
            out["tokens"][s, n] = x
            out["logprob"][s, n] = np.log(p[x])
            n += 1
        out["accepted"][s] = n
        y = None
        if live:
            if t_target == 0.0:
                y = int(np.argmax(target[s, n]))
            else:
                y, ratio = race(weight, noise[s])
                out["margin"][s] = min(out["margin"][s], ratio - 1.0)
                out["nonfinite"] |= y is None
        if y is None:
            out["logprob"][s, n] = np.nan
        else:
            out["tokens"][s, n] = y
            z = target[s, n]
            a = (z - z.max()) / t
            out["logprob"][s, n] = a[y] - np.log(np.exp(a).sum())
    return out


def embed(w, tokens, scale=1.0, ignore_index=-100):
    w = as_f64(w)
    h = np.zeros((len(tokens), w.shape[1]))
    for n, t in enumerate(tokens):
        if t != ignore_index and 0 <= t < len(w):
            h[n] = w[t] * scale
    return h


def embed_grad(d_h, tokens, vocab, scale=1.0, ignore_index=-100):
    """(d_w, sum of the absolute values that were added, number of rows added)."""
    d_h = as_f64(d_h)
    d_w, size, count = (np.zeros((vocab, d_h.shape[1])), np.zeros((vocab, d_h.shape[1])),
                        np.zeros(vocab, np.int64))
    for n, t in enumerate(tokens):
        if t != ignore_index and 0 <= t < vocab:
            d_w[t] += d_h[n] * scale
            size[t] += np.abs(d_h[n] * scale)
            count[t] += 1
    return d_w, size, count


def rms_norm(x, weight, residual=None, eps=1e-6, weight_offset=0.0):
    s = as_f64(x) if residual is None else as_f64(x) + as_f64(residual)
    r = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return s * r * (as_f64(weight) + weight_offset), s


def rms_norm_grad(s, weight, d_h, d_sum=None, eps=1e-6, weight_offset=0.0):
    """dict(d_x, d_weight, x_size, w_size): the gradients, and the sums of the
    absolute values of what each is made of."""
    s, d_h = as_f64(s), as_f64(d_h)
    r = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    g = d_h * (as_f64(weight) + weight_offset)
    c = r ** 3
    d_x = r * g - s * c * (g * s).mean(axis=1, keepdims=True)
    size = np.abs(r * g) + np.abs(s) * c * np.abs(g * s).mean(axis=1, keepdims=True)
    if d_sum is not None:
        d_x = d_x + as_f64(d_sum)
        size = size + np.abs(as_f64(d_sum))
    return {"d_x": d_x, "x_size": size, "d_weight": (d_h * s * r).sum(axis=0),
            "w_size": np.abs(d_h * s * r).sum(axis=0)}
