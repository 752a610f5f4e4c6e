"""The float64 oracle of the operators around a layer's Linears: its gradients against central differences of its forward
forms, its scales against their definition."""

import numpy as np
import pytest

from oracle import layer


def difference(f, x, d, step=1e-6):
    """Derivative of f at x in direction d."""
    return (f(x + step * d) - f(x - step * d)) / (2 * step)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (4, 130)])
def test_norm_gradient(rows, cols, residual):
    rng = np.random.default_rng(cols)
    x, r, dy, dh = (rng.normal(size=(rows, cols)) for _ in range(4))
    w, eps = rng.normal(1, 0.3, cols), 1e-2
    r, dh = (r, dh) if residual else (None, None)

    def value(x, w):
        h, _, y = layer.rmsnorm(x, r, w, eps)
        return (y * dy).sum() + (0 if dh is None else (h * dh).sum())

    h, rstd, _ = layer.rmsnorm(x, r, w, eps)
    dx, dw = layer.rmsnorm_grad(dy, h, w, rstd, dh)
    for _ in range(3):
        d, e = rng.normal(size=x.shape), rng.normal(size=cols)
        assert difference(lambda v: value(v, w), x, d) == pytest.approx((dx * d).sum(), rel=1e-6, abs=1e-8)
        assert difference(lambda v: value(x, v), w, e) == pytest.approx((dw * e).sum(), rel=1e-6, abs=1e-8)


def test_combine_gradient():
    rng = np.random.default_rng(1)
    tokens, topk, rows, cols = 7, 3, 20, 9
    pos = rng.permutation(rows + 3)[: tokens * topk].reshape(tokens, topk).astype(np.int64)
    pos[pos >= rows] = -1
    y, w = rng.normal(size=(rows, cols)), rng.normal(size=(tokens, topk))
    dout = rng.normal(size=(tokens, cols))
    dy, dw, _ = layer.combine_grad(dout, y, pos, w)
    value = lambda y, w: (layer.combine(y, pos, w, None)[0] * dout).sum()  # noqa: E731
    d, e = rng.normal(size=y.shape), rng.normal(size=w.shape)
    assert difference(lambda v: value(v, w), y, d) == pytest.approx((dy * d).sum(), rel=1e-7)
    assert difference(lambda v: value(y, v), w, e) == pytest.approx((dw * e).sum(), rel=1e-7)


def test_dispatch_gradient_is_the_unweighted_combine():
    rng = np.random.default_rng(2)
    pos = np.array([[0, 3], [-1, 1], [4, -1]])
    src = np.array([0, 1, -1, 0, 2, -2])
    x, drows = rng.normal(size=(3, 4)), rng.normal(size=(6, 4))
    drows[5] = 0
    rows = layer.dispatch(x, pos, src, 6, 0.0)
    assert (rows[2] == 0).all() and np.array_equal(rows[4], x[2])
    d = rng.normal(size=x.shape)
    assert (layer.dispatch(d, pos, src, 6, 0.0) * drows).sum() == pytest.approx((layer.combine(drows, pos, None, None)[0] * d).sum())


@pytest.mark.parametrize("amax", [448.0, 448.0000001, 447.999, 1e-3, 2.0 ** -140, 1.75 * 2.0 ** 20, 1.75 * 2.0 ** 20 * (1 + 2 ** -50)])
def test_power_of_two_scale(amax):
    s = float(layer.scale(np.array(amax), True))
    assert amax <= 448 * s and (amax > 448 * s / 2 or s == 2.0 ** -127)


def test_scale_of_zeros():
    assert layer.scale(np.zeros(1), False)[0] == 0 and layer.scale(np.zeros(1), True)[0] == 2.0 ** -127
