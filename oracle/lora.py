"""Low-rank adapters beside a shared projection, and their gradient, in FP64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Definition: include/nvfp4_moe.h, "Low-rank adapters beside a shared projection".  Adapter by
adapter; shares no code with the kernels.  Pinned by ``tests/test_oracle_lora.py``.
"""

import numpy as np


def _rows(ids, L):
    return [np.flatnonzero(np.asarray(ids) == a) for a in range(L)]


def add(y, x, down, up, scale, ids):
    """(y + scale_a B_a (A_a x), h), row by row the adapter ids[t]; negative ids and those past the last: none."""
    out, h = np.array(y, np.float64), np.zeros((x.shape[0], down.shape[1]))
    for a, rows in enumerate(_rows(ids, down.shape[0])):
        h[rows] = x[rows] @ down[a].T
        out[rows] += scale[a] * (h[rows] @ up[a].T)
    return out, h


def backward(dy, x, h, down, up, scale, ids):
    """(dx, ddown, dup, dh)."""
    dx, dh = np.zeros((x.shape[0], down.shape[2])), np.zeros((x.shape[0], down.shape[1]))
    ddown, dup = np.zeros(down.shape), np.zeros(up.shape)
    for a, rows in enumerate(_rows(ids, down.shape[0])):
        dh[rows] = scale[a] * (dy[rows] @ up[a])
        dx[rows] = dh[rows] @ down[a]
        ddown[a] = dh[rows].T @ x[rows]
        dup[a] = scale[a] * (dy[rows].T @ h[rows])
    return dx, ddown, dup, dh
