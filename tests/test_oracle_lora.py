"""The FP64 adapters of the oracle: a token at a time, and the gradient against differences."""

import numpy as np

from oracle import lora as O


def make(T=7, K=6, N=5, R=3, L=4, seed=0):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    return n((T, N)), n((T, K)), n((L, R, K)), n((L, N, R)), n(L), np.array([2, -1, 0, 2, 3, 9, 0])[:T]


def test_by_token():
    y, x, down, up, scale, ids = make()
    out, h = O.add(y, x, down, up, scale, ids)
    for t, a in enumerate(ids):
        if 0 <= a < 4:
            assert np.allclose(h[t], down[a] @ x[t]) and np.allclose(out[t], y[t] + scale[a] * up[a] @ (down[a] @ x[t]))
        else:
            assert np.array_equal(out[t], y[t]) and not h[t].any()


def test_gradient():
    y, x, down, up, scale, ids = make(seed=1)
    dy = np.random.default_rng(2).standard_normal(y.shape)
    _, h = O.add(y, x, down, up, scale, ids)
    dx, ddown, dup, _ = O.backward(dy, x, h, down, up, scale, ids)
    step = 1e-6

    def total(**kw):
        v = dict(x=x, down=down, up=up)
        v.update(kw)
        return (dy * O.add(y, v["x"], v["down"], v["up"], scale, ids)[0]).sum()

    for name, at, grad in (("x", x, dx), ("down", down, ddown), ("up", up, dup)):
        for i in np.ndindex(at.shape):
            a, b = at.copy(), at.copy()
            a[i] += step
            b[i] -= step
            assert abs(grad[i] - (total(**{name: a}) - total(**{name: b})) / (2 * step)) < 1e-7
