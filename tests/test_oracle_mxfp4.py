"""Pins of the MXFP4 and routing oracles: values worked out by hand, the nearest-code definition in exact rational
arithmetic, gradients against differences."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import moe, mxfp4


def test_codes_by_hand():
    y = np.array([0.0, -0.0, 0.25, 0.2500001, -0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 7.9, -6.0, 0.1])
    #            0    -0    tie->0  0.5     tie->1(-) tie->1 tie->2 tie->2 tie->4 tie->4 6   sat  -6   0
    assert mxfp4.decode(mxfp4.encode(y)).tolist() == [0, 0, 0, 0.5, -1, 1, 2, 2, 4, 4, 6, 6, -6, 0]
    assert mxfp4.encode(y)[1] == 8 and mxfp4.encode(np.array([-0.2]))[0] == 8       # sign of zero kept


def test_codes_against_rational_search():
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.normal(0, 3, 500), np.arange(-64, 65) / 8.0, np.nextafter(np.arange(0, 49) / 8.0, 9)])
    for v, c in zip(y, mxfp4.encode(y)):
        d = [abs(abs(Fraction(v)) - Fraction(g)) for g in mxfp4.GRID]
        best = [i for i in range(8) if d[i] == min(d)]
        want = best[0] if len(best) == 1 else [i for i in best if i % 2 == 0][0]
        assert (c & 7) == want and (c >> 3) == int(np.signbit(v))


def test_scales_by_hand():
    assert mxfp4.tile_exponent(6.0, False) == 0 and mxfp4.tile_exponent(4.0, False) == 0
    assert mxfp4.tile_exponent(7.9, False) == 0 and mxfp4.tile_exponent(7.9, True) == 1
    assert mxfp4.tile_exponent(6.0, True) == 0 and mxfp4.tile_exponent(8.0, False) == 1
    assert mxfp4.tile_exponent(2.0 ** -140, False) == -127 and mxfp4.tile_exponent(0.0, True) == -127


def test_layout_and_tail():
    x = np.zeros((2, 300))
    x[0, 0], x[0, 1], x[1, 299] = 4.0, -6.0, 1.5
    q, s = mxfp4.quantise(x)
    assert q.shape == (2, 256) and s.shape == (2, 2, 8)
    assert q[0, 0] == (6 | (15 << 4)) and s[0, 0, 0] == 127
    assert q[1, 149] >> 4 == 7 and s[1, 1, 1] == 125          # 1.5 = 6 * 2^-2
    assert np.array_equal(mxfp4.values(q, s, 300), x)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_tile_with_a_nonfinite_value(bad):
    x = np.ones((1, 64))
    x[0, 40] = bad
    q, s = mxfp4.quantise(x)
    assert s[0, 0, 1] == 255 and not q[0, 16:32].any()
    v = mxfp4.values(q, s, 64)
    assert (v[0, :32] == 1).all() and np.isnan(v[0, 32:]).all()


@pytest.mark.parametrize("nosat", [False, True])
def test_error_bound(nosat):
    # half a step: 2^-2 of the value in the normal range (E2M1 has one mantissa bit), 0.25 * scale below it, and
    # without nosat up to 2 * scale where the largest elements saturate
    x = np.random.default_rng(1).standard_t(3, (16, 512))
    q, s = mxfp4.quantise(x, nosat)
    v = mxfp4.values(q, s, 512)
    scale = np.repeat(np.exp2(s.transpose(1, 0, 2).reshape(16, -1) - 127.0), 32, 1)
    bound = np.maximum(np.abs(x) / 4, scale / 4)
    if not nosat:
        bound = np.where(np.abs(x) > 6 * scale, 2 * scale, bound)
    assert (np.abs(v - x) <= bound).all()


def test_plan_by_hand():
    idx = np.array([[1, 0], [1, 5], [-1, 1]], np.int32)
    counts, off, src, pos = moe.plan(idx, 3, 2, 9)
    assert counts.tolist() == [1, 3, 0] and off.tolist() == [0, 2, 6, 6]
    assert src.tolist() == [0, -1, 0, 1, 2, -1, -2, -2, -2] and pos.tolist() == [[2, 0], [3, -1], [-1, 4]]


def test_balance_by_hand():
    # two tokens, two experts, equal scores: f = (2 * 2 / (1 * 2), 0), P = (1/2, 1/2): loss = coef
    loss, counts, real = moe.balance(np.zeros((2, 2)), np.array([[0], [0]]), 0.5, "softmax", [0, 2])
    assert loss == pytest.approx(0.5) and counts.tolist() == [[2, 0]] and real.tolist() == [2]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(score):
    rng = np.random.default_rng(2)
    x = rng.normal(size=(9, 5))
    idx = rng.integers(-1, 6, (9, 2))
    off = [1, 4, 4, 8]
    g = moe.balance_grad(1.7, x, idx, 0.3, score, off)
    h = 1e-5
    for t in range(9):
        for e in range(5):
            up, dn = x.copy(), x.copy()
            up[t, e] += h
            dn[t, e] -= h
            d = 1.7 * (moe.balance(up, idx, 0.3, score, off)[0] - moe.balance(dn, idx, 0.3, score, off)[0]) / (2 * h)
            assert abs(d - g[t, e]) < 1e-9
