"""The operators around a layer's Linears in float64, as their formulas say: RMS norm after the residual's addition with
its gradient, tokens to the rows of a dispatch plan and back with the gates' weights, and the gradient. Slow and plain;
shares nothing with the library."""

import numpy as np


def rmsnorm(x, residual, weight, eps):
    """(h, rstd, y) of float64 x [rows, cols], residual the same or None."""
    h = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((h * h).sum(1) / h.shape[1] + eps)
    return h, rstd, h * rstd[:, None] * weight


def rmsnorm_grad(dy, h, weight, rstd, dh):
    """(dx, dweight) for given rstd; dx is the gradient of everything that was added up to h."""
    hat = h * rstd[:, None]
    g = dy * weight
    dx = rstd[:, None] * (g - hat * (g * hat).mean(1, keepdims=True))
    return dx if dh is None else dx + dh, (dy * hat).sum(0)


def scale(amax, pow2):
    """Scale of an E4M3 tile of largest magnitude amax (float64)."""
    if not pow2:
        return amax / 448.0
    with np.errstate(divide="ignore"):
        k = np.ceil(np.log2(np.where(amax > 0, amax, 1.0) / 448.0))
    k = np.where(amax > 448.0 * np.exp2(k), k + 1, np.where(amax <= 448.0 * np.exp2(k - 1), k - 1, k))    # log2's own rounding
    return np.exp2(np.where(amax > 0, np.clip(k, -127, 127), -127))


def dispatch(x, pos, src, rows, unused):
    """Rows of a plan: those with a token, zeros, and `unused` where src is -2."""
    out = np.zeros((rows, x.shape[1]), x.dtype)
    out[src == -2] = unused
    for t in range(pos.shape[0]):
        for r in pos[t]:
            if 0 <= r < rows:
                out[r] = x[t]
    return out


def combine(y, pos, weight, base):
    """Sum of a token's rows, weighted; and the sum of the terms' magnitudes."""
    out = np.zeros((pos.shape[0], y.shape[1]))
    mag = np.zeros_like(out)
    for t in range(pos.shape[0]):
        if base is not None:
            out[t] += base[t]
            mag[t] += np.abs(base[t])
        for j, r in enumerate(pos[t]):
            if 0 <= r < len(y):
                term = y[r] if weight is None else weight[t, j] * y[r]
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


def combine_grad(dout, y, pos, weight):
    """(dy with zeros where there is no token, dweight, sum of the dot products' magnitudes)."""
    dy = np.zeros_like(y)
    dw = np.zeros(pos.shape)
    mag = np.zeros(pos.shape)
    for t in range(pos.shape[0]):
        for j, r in enumerate(pos[t]):
            if 0 <= r < len(y):
                dy[r] = weight[t, j] * dout[t]
                dw[t, j] = dout[t] @ y[r]
                mag[t, j] = np.abs(dout[t]) @ np.abs(y[r])
    return dy, dw, mag
