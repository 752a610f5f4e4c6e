"""Helpers of the MXFP4 tests: seeded inputs, the accumulation bound, comparison with the oracle. Not a test module."""

from __future__ import annotations

import numpy as np

from oracle import mxfp4

DTYPES = ("bfloat16", "float16", "float32")


def torch_dtype(name):
    import torch
    return getattr(torch, name)


def matrix(seed, rows, cols, dtype="bfloat16", std=1.0, ld=None, device="cuda"):
    """A seeded [rows, cols] tensor with outliers, one zero tile and one row of tiny values, as a view of rows `ld` long."""
    import torch
    rng = np.random.default_rng(seed)
    x = rng.normal(0, std, (rows, cols))
    x = np.where(rng.random(x.shape) < 0.01, x * 40, x)
    x[rows // 2, : min(32, cols)] = 0.0
    x[rows // 3] *= 2.0 ** -10
    t = torch.full((rows, ld or cols), float("nan"), dtype=torch_dtype(dtype), device=device)   # poison between rows
    t[:, :cols] = torch.from_numpy(x).to(torch_dtype(dtype))
    return t[:, :cols]


def f64(t):
    return t.detach().to("cpu").double().numpy()


def accumulation_bound(k, ab):
    """|fp32 accumulation - exact| for sums of exact products: at most k additions (tiles, blocks, waves), each off by
    at most one unit in the last place (2^-23) of a partial sum that never exceeds sum |a||b|."""
    return (k + 64) * 2.0 ** -23 * ab


def check_product(out, va, vb, k, dtype):
    """out [m, n] (host float64) against the product of the operands' values [m, k], [n, k]."""
    exact = va @ vb.T
    ab = np.abs(va) @ np.abs(vb).T
    tol = accumulation_bound(k, ab)
    if dtype == "bfloat16":
        tol = tol + 2.0 ** -8 * (np.abs(exact) + tol) + 2.0 ** -134   # half a step of bf16 (and of its subnormals)
    bad = ~(np.abs(out - exact) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}"


def codes(q, s, k):
    """Values of device codes and scales."""
    return mxfp4.values(q.cpu().numpy(), s.cpu().numpy(), k)


def operand(seed, rows, k, device="cuda"):
    """Random codes and scales in the packed layout (the oracle's), on the device, with their values."""
    import torch
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, k)) * np.exp2(rng.integers(-3, 4, (rows, 1)))
    q, s = mxfp4.quantise(x)
    return torch.from_numpy(q).to(device), torch.from_numpy(s).to(device), mxfp4.values(q, s, k)
