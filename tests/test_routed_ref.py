"""The references of the routed layers: their gradients against differences (CPU, 64 bits)."""
import numpy as np

from tests import routed_ref as R


def difference(f, x, dout, step=1e-5):
    """Central differences of <dout, f(x)> along every element of x."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        at = x[i]
        x[i] = at + step
        up = (dout * f()).sum()
        x[i] = at - step
        g[i] = (up - (dout * f()).sum()) / (2 * step)
        x[i] = at
    return g


def test_plan():
    offsets, rows, src = R.plan(np.array([[2, 0], [2, 9], [-1, 2], [0, 3]]), 4, 4)
    assert offsets.tolist() == [0, 4, 4, 8, 12]
    assert rows.tolist() == [[4, 0], [5, -1], [-1, 6], [1, 8]]
    assert src.tolist() == [1, 6, -1, -1, 0, 2, 5, -1, 7, -1, -1, -1] + [-1] * 8


def test_combine():
    rng = np.random.default_rng(0)
    ids = rng.integers(-1, 3, (5, 2))
    _, rows, src = R.plan(ids, 3, 2)
    y, w, res, dout = rng.normal(size=(len(src), 4)), rng.normal(size=rows.shape), rng.normal(size=(5, 4)), rng.normal(size=(5, 4))
    dy, dw, _ = R.combine_grad(dout, y, rows, src, w)
    f = lambda: R.combine(y, rows, w, res)[0]
    assert np.allclose(dy, difference(f, y, dout), atol=1e-9) and np.allclose(dw, difference(f, w, dout), atol=1e-9)


def test_adapters():
    rng = np.random.default_rng(1)
    ids = np.array([1, -1, 0, 1, 3, 1])
    x, A, B = rng.normal(size=(6, 5)), rng.normal(size=(4, 2, 5)), rng.normal(size=(4, 3, 2))
    scale, base, dy = rng.normal(size=4), rng.normal(size=(6, 3)), rng.normal(size=(6, 3))
    (dx, dA, dB), _ = R.adapters_grad(dy, x, A, B, ids, scale, np.zeros_like(x))
    f = lambda: R.adapters(x, A, B, ids, scale, base)[0]
    for g, v in ((dx, x), (dA, A), (dB, B)):
        assert np.allclose(g, difference(f, v, dy), atol=1e-8)
