"""MXFP4 (OCP Microscaling Formats v1.0: E2M1 elements, one E8M0 scale per 32) from its definition, in float64.

Test infrastructure, sharing nothing with the HIP path. A tile is 32 consecutive elements of the last axis; its
scale is 2^e with e = floor(log2(amax)) - 2 (or, nosat, the smallest e with amax <= 6 * 2^e), e >= -127, -127 for an
all-zero tile; a tile with a NaN or an infinity has the scale byte 0xFF and zero codes. Codes are the nearest E2M1
value of x * 2^-e, ties to the even code, saturated, sign kept.
"""

from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
NAN_BYTE = 255


def encode(y: np.ndarray) -> np.ndarray:
    """E2M1 codes of float64 values already divided by their scale."""
    a = np.abs(y)
    d = np.abs(a[..., None] - GRID)
    best = d.min(-1, keepdims=True)
    near = d == best                                   # one candidate, or the two neighbours of a midpoint
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1, keepdims=True) & (near.sum(-1, keepdims=True) > 1), even, near)
    code = pick.argmax(-1).astype(np.uint8)
    return code | (np.signbit(y).astype(np.uint8) << 3)


def decode(code: np.ndarray) -> np.ndarray:
    return GRID[code & 7] * np.where(code & 8, -1.0, 1.0)


def tile_exponent(amax: float, nosat: bool) -> int:
    """e of a finite tile."""
    if amax == 0:
        return -127
    m, ex = np.frexp(amax)                              # amax = m * 2^ex, m in [0.5, 1)
    e = int(ex) - 3
    if nosat and amax > 6.0 * 2.0 ** e:
        e += 1
    return max(e, -127)


def quantise(x: np.ndarray, nosat: bool = False):
    """x float64 [rows, k] -> (codes uint8 [rows, chunks * 128], scales uint8 [chunks, rows, 8]): the packed layout,
    padded to whole chunks of 256 elements."""
    rows, k = x.shape
    chunks = -(-k // 256)
    t = np.zeros((rows, chunks * 256))
    t[:, :k] = x
    t = t.reshape(rows, chunks * 8, 32)
    with np.errstate(invalid="ignore"):
        bad = ~np.isfinite(t).all(-1)
    t = np.where(bad[..., None], 0.0, t)
    amax = np.abs(t).max(-1)
    m, ex = np.frexp(amax)
    e = ex.astype(np.int64) - 3
    if nosat:
        e += amax > 6.0 * np.exp2(e.astype(np.float64))
    e = np.where(amax == 0, -127, np.maximum(e, -127))
    code = np.concatenate([encode(p * np.exp2(-ee.astype(np.float64))[..., None])
                           for p, ee in zip(np.array_split(t, max(1, t.size >> 20)), np.array_split(e, max(1, t.size >> 20)))])
    code = np.where(bad[..., None], 0, code).astype(np.uint8).reshape(rows, chunks * 256)
    byte = np.where(bad, NAN_BYTE, e + 127).astype(np.uint8)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), \
        np.ascontiguousarray(byte.reshape(rows, chunks, 8).transpose(1, 0, 2))


def values(q: np.ndarray, s: np.ndarray, k: int) -> np.ndarray:
    """float64 [rows, k] that packed codes and scales stand for."""
    rows = q.shape[0]
    code = np.empty((rows, q.shape[1] * 2), np.uint8)
    code[:, 0::2], code[:, 1::2] = q & 15, q >> 4
    byte = s.transpose(1, 0, 2).reshape(rows, -1).astype(np.float64)
    scale = np.where(byte == NAN_BYTE, np.nan, np.exp2(byte - 127))
    return (decode(code).reshape(rows, -1, 32) * scale[..., None]).reshape(rows, -1)[:, :k]
