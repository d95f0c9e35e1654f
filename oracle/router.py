"""Choosing experts from router scores, and the logits' gradient (oracle; test
infrastructure only).  This library's own addition (mgemm.h states it): softmax
or sigmoid scores, a bias for the choice, groups, top-k, renormalized weights.
Float64 numpy, one token at a time.
"""

import numpy as np

MASKED = -3.3e38


def _scores(l, scoring):
    off = l <= MASKED
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-l))
    else:
        m = np.max(l)
        e = np.exp(l - (0.0 if m <= MASKED else m))
        e = np.where(off, 0.0, e)
        s = e / e.sum() if e.sum() != 0 else e
    return np.where(off, 0.0, s), off


def _order(keys):
    """Indices by key descending, ties by index; a key is (class, value), a NaN the largest."""
    return sorted(range(len(keys)), key=lambda i: (-keys[i][0], -np.inf if np.isnan(keys[i][1]) else -keys[i][1], i))


def choose(l, k, scoring, bias=None, n_group=1, topk_group=1, group_top=1):
    """ids of one token's experts (logits l float64 [E]), best first."""
    E = len(l)
    s, off = _scores(l, scoring)
    c = s + bias if bias is not None else s
    if scoring == "softmax" and bias is None:
        c = l
    terms = s if scoring == "softmax" and bias is None and group_top == 2 else c
    allowed = np.ones(E, dtype=bool)
    if n_group > 1:
        gs = E // n_group
        scores = []
        for g in range(n_group):
            members = [terms[e] for e in range(g * gs, (g + 1) * gs) if not off[e]]
            members.sort(key=lambda v: np.inf if np.isnan(v) else v, reverse=True)
            scores.append((1, sum(members[:group_top])) if members else (0, 0.0))
        for g in _order(scores)[topk_group:]:
            allowed[g * gs:(g + 1) * gs] = False
    keys = [(2 if allowed[e] and not off[e] else 1 if allowed[e] else 0, c[e] if allowed[e] and not off[e] else 0.0)
            for e in range(E)]
    return _order(keys)[:k]


def weights(l, ids, scoring, renormalize=True, scale=1.0):
    s, _ = _scores(l, scoring)
    r = s[ids]
    if renormalize:
        r = r / r.sum() if r.sum() != 0 else np.zeros_like(r)
    return scale * r


def route(logits, k, scoring, bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0):
    logits = np.asarray(logits, dtype=np.float64)
    ids = np.array([choose(l, k, scoring, bias, n_group, topk_group, group_top) for l in logits]).reshape(-1, k)
    w = np.array([weights(l, i, scoring, renormalize, scale) for l, i in zip(logits, ids)]).reshape(-1, k)
    return w, ids


def route_grad(g, logits, ids, scoring, renormalize=True, scale=1.0):
    """dL/dlogits from dL/dw = g, by the chain rule through the picked scores."""
    logits = np.asarray(logits, dtype=np.float64)
    out = np.zeros_like(logits)
    for t, l in enumerate(logits):
        s, off = _scores(l, scoring)
        r = s[ids[t]]
        if renormalize:
            S = r.sum()
            dr = scale * (g[t] / S - (g[t] * r).sum() / S ** 2) if S != 0 else np.zeros_like(r)
        else:
            dr = scale * g[t]
        ds = np.zeros(len(l))
        ds[ids[t]] = dr
        if scoring == "sigmoid":
            out[t] = ds * s * (1 - s)
        else:  # renormalized weights do not change with a common factor of the scores: sum dr r is 0
            out[t] = s * (ds - (0.0 if renormalize else (ds * s).sum()))
    return out
