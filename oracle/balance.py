"""The balance loss of a router (oracle; test infrastructure only).

Not on the source pages.  Over the n counted tokens of a sequence, c_e of whose k n picks are
expert e: L_s = sum_e (E c_e / (k n)) (sum_t p_te / n), p a token's softmax or its sigmoids
over their sum, 0 for experts that are off; the loss is scale times the mean of L_s over the
sequences with tokens.  The counts are constant in the gradient:
  dL_s/dp_te = a_e = E c_e / (k n^2),  dL/dl = p (a - sum p a)  [sigmoid: times 1 - s,
which is 1 / (1 + e^l)].
Float64 numpy, loops over sequences and tokens.
"""

import numpy as np

OFF = -3.3e38


def scores(l, scoring):
    """(p, s) of one token's logits: the normalized and the raw scores."""
    l = np.asarray(l, dtype=np.float64)
    on = ~(l <= OFF)
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            s = np.where(on, 1.0 / (1.0 + np.exp(-l)), 0.0)
    else:
        s = np.where(on, np.exp(l - (np.max(l[on]) if on.any() else 0.0)), 0.0)
    total = s.sum()
    return (s / total if total != 0 else np.zeros_like(s)), s


def score_rest(l, scoring):
    """ds/dl / s of one token's logits: 1 - s for sigmoids without cancellation, else 1."""
    l = np.asarray(l, dtype=np.float64)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(l)) if scoring == "sigmoid" else np.ones_like(l)


def _tokens(T, offsets, mask):
    bounds = [0, T] if offsets is None else [int(o) for o in offsets]
    return [[t for t in range(a, b) if mask is None or mask[t]] for a, b in zip(bounds[:-1], bounds[1:])]


def counts(ids, E, rows):
    c = np.zeros(E, dtype=np.int64)
    for t in rows:
        for e in ids[t]:
            if 0 <= e < E:
                c[e] += 1
    return c


def balance(logits, ids, scoring, scale=1.0, offsets=None, mask=None):
    """(loss, counts int64 [S, E])."""
    T, E = logits.shape
    k = ids.shape[1]
    every, losses = [], []
    for rows in _tokens(T, offsets, mask):
        c = counts(ids, E, rows)
        every.append(c)
        if rows:
            n = len(rows)
            p = sum(scores(logits[t], scoring)[0] for t in rows)
            losses.append(np.sum(E * c / (k * n) * (p / n)))
    return scale * (np.mean(losses) if losses else 0.0), np.stack(every)


def balance_grad(grad_loss, logits, ids, scoring, scale=1.0, offsets=None, mask=None):
    """(dL/dlogits [T, E], the sizes of the terms that cancel in it)."""
    T, E = logits.shape
    k = ids.shape[1]
    grad, size = np.zeros((T, E)), np.zeros((T, E))
    groups = _tokens(T, offsets, mask)
    present = sum(bool(r) for r in groups)
    for rows in groups:
        if not rows:
            continue
        a = grad_loss * scale / present * E * counts(ids, E, rows) / (k * len(rows) ** 2)
        for t in rows:
            p, _ = scores(logits[t], scoring)
            grad[t] = p * (a - np.sum(p * a)) * score_rest(logits[t], scoring)
            size[t] = p * (np.abs(a) + np.sum(p * np.abs(a)))
    return grad, size
