"""Routing of given logits (scores, bias, groups, top-k, renormalisation) and its gradient, in FP64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Definition: include/nvfp4_moe.h, "Routing of given logits".  Row by row, by sorting; shares no
code with the kernels.  Pinned by ``tests/test_oracle_route_topk.py``.
"""

import numpy as np


def scores(logits, score):
    """s [T, E]: softmax or sigmoid; 0 where the logit is -inf or NaN."""
    l = np.asarray(logits, np.float64)
    masked = ~(l > -np.inf)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-np.where(masked, 0.0, l)))
        return np.where(masked, 0.0, s)
    out = np.zeros_like(l)
    for t in range(l.shape[0]):
        live = ~masked[t]
        if live.any():
            m = l[t, live].max()
            z = np.where(l[t, live] == m, 1.0, np.exp(np.where(l[t, live] == m, 0.0, l[t, live] - m)))
            out[t, live] = z / z.sum()
    return out


def order_values(logits, score, bias=None):
    """o [T, E]; -inf for what is chosen last."""
    l = np.asarray(logits, np.float64)
    if bias is None:
        o = np.where(l > -np.inf, l, -np.inf)
    else:
        o = np.where(l > -np.inf, scores(l, score) + np.asarray(bias, np.float64)[None, :], -np.inf)
    return np.where(o > -np.inf, o, -np.inf)


def group_scores(logits, score, bias, n_group, group_score):
    o = order_values(logits, score, bias)
    T, E = o.shape
    if group_score == "max":
        return o.reshape(T, n_group, E // n_group).max(-1)
    v = o if bias is not None else np.where(o > -np.inf, scores(logits, score), -np.inf)
    v = -np.sort(-v.reshape(T, n_group, E // n_group), axis=-1)[..., :2]
    two = v[..., 0] + (np.where(v[..., 1] > -np.inf, v[..., 1], 0.0) if v.shape[-1] > 1 else 0.0)
    return two


def route(logits, k, score="softmax", bias=None, n_group=1, topk_group=1, group_score="max", renormalize=True,
          scale=1.0):
    """(ids int32 [T, k], weights float64 [T, k])."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    o = order_values(l, score, bias)
    allowed = np.ones((T, E), bool)
    if n_group > 1:
        gs = group_scores(l, score, bias, n_group, group_score)
        keep = np.zeros((T, n_group), bool)
        for t in range(T):
            keep[t, np.lexsort((np.arange(n_group), -gs[t]))[:topk_group]] = True
        allowed = np.repeat(keep, E // n_group, axis=1)
    ids = np.empty((T, k), np.int32)
    for t in range(T):
        # allowed before not allowed, larger order value first, lower id first
        ids[t] = np.lexsort((np.arange(E), -o[t], ~allowed[t]))[:k]
    return ids, weights(l, ids, score, renormalize, scale)


def weights(logits, ids, score, renormalize, scale):
    """w [T, k] of given ids."""
    l = np.asarray(logits, np.float64)
    i = np.asarray(ids, np.int64)
    if score == "softmax" and renormalize:
        # the chosen scores over their sum = the softmax over the chosen (which does not underflow)
        return scores(np.take_along_axis(l, i, 1), score) * scale
    s = np.take_along_axis(scores(l, score), i, 1)
    if renormalize:
        total = s.sum(1, keepdims=True)
        s = np.where(total > 0, s / np.where(total > 0, total, 1.0), 0.0)
    return s * scale


def backward(logits, ids, dw, score, renormalize, scale):
    """Gradient of sum(dw * w) with respect to the logits [T, E], FP64, from the Jacobian of each
    row's scores (softmax: diag(s) - s s^T; sigmoid: diag(s (1 - s))).  The renormalised softmax is
    the softmax over the chosen, so there only their logits take part."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    out = np.zeros((T, E))
    full = scores(l, score)
    for t in range(T):
        i = np.asarray(ids[t], np.int64)
        g = np.asarray(dw[t], np.float64) * scale
        if score == "softmax":
            if renormalize:
                q = scores(l[t:t + 1, i], score)[0]
                out[t, i] = q * (g - (g * q).sum())
            else:
                s, ds = full[t], np.zeros(E)
                np.add.at(ds, i, g)
                out[t] = s * (ds - (ds * s).sum())
            continue
        s = full[t, i]
        if renormalize:
            total = s.sum()
            if total <= 0:
                continue
            # d(s_j / S) / ds_c = [j = c] / S - s_j / S^2
            g = g / total - (g * s).sum() / total ** 2
        np.add.at(out[t], i, g * s * (1.0 - s))
    return out
