"""A router's balance loss over packed sequences and its gradient, in FP64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Definition: include/nvfp4_moe.h, "Balance loss of a router".  Row by row; shares no code with the
kernels.  Pinned by ``tests/test_oracle_balance.py``.
"""

import numpy as np


def probabilities(row, score):
    """p [E] of one row of logits; 0 where the logit is -inf or NaN."""
    l = np.asarray(row, np.float64)
    p = np.zeros_like(l)
    live = np.flatnonzero(l > -np.inf)
    if live.size == 0:
        return p
    z = l[live]
    m = z.max()
    if score == "softmax":
        if m == np.inf:
            e = (z == np.inf).astype(np.float64)
        else:
            e = np.exp(z - m)
    else:
        if m < -709.0:
            return p
        # log sigmoid(z) = min(z, 0) - log(1 + e^-|z|), relative to its largest
        log_s = np.minimum(z, 0.0) - np.log1p(np.exp(-np.abs(z)))
        e = np.exp(log_s - log_s.max())
    p[live] = e / e.sum()
    return p


def members(T, mask, offsets):
    """Rows that count, for each sequence."""
    cuts = [0, T] if offsets is None else [int(o) for o in offsets]
    return [[t for t in range(a, b) if mask is None or mask[t]] for a, b in zip(cuts[:-1], cuts[1:])]


def loss(logits, ids, score="softmax", mask=None, offsets=None):
    """(loss [S], counts [S, E], probs [S, E], tokens [S])."""
    T, E = logits.shape
    k = ids.shape[1]
    out = []
    for rows in members(T, mask, offsets):
        n = len(rows)
        counts, mean = np.zeros(E, np.int64), np.zeros(E)
        for t in rows:
            mean += probabilities(logits[t], score)
            for e in ids[t]:
                if 0 <= e < E:
                    counts[e] += 1
        if n:
            mean /= n
        out.append((E * float((counts * mean).sum()) / (k * n) if n else 0.0, counts, mean, n))
    return tuple(np.array([o[i] for o in out]) for i in range(4))


def backward(logits, k, counts, tokens, dloss, score="softmax", mask=None, offsets=None):
    """(gradient [T, E], the sum of the magnitudes of the terms it is the difference of [T, E])."""
    T, E = logits.shape
    d, size = np.zeros((T, E)), np.zeros((T, E))
    for s, rows in enumerate(members(T, mask, offsets)):
        n = float(tokens[s])
        if n == 0:
            continue
        g = float(dloss[s]) * E * np.asarray(counts[s], np.float64) / (k * n * n)
        for t in rows:
            p = probabilities(logits[t], score)
            d[t] = p * (g - (g * p).sum())
            size[t] = p * (np.abs(g) + (np.abs(g) * p).sum())
            if score == "sigmoid":
                l = np.where(p > 0, np.asarray(logits[t], np.float64), 0.0)
                with np.errstate(over="ignore"):
                    rest = 1.0 / (1.0 + np.exp(l))
                d[t] *= rest
                size[t] *= rest
    return d, size
