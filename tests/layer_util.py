"""Helpers of the tests of the operators around a layer's Linears. Not a test module.

Tolerances count roundings. U is half a step of float32 relative to the value. A lane adds up at most 64 elements of a
row one after the other, and its sum goes through at most 16 more additions (lanes of a wave, waves of a workgroup), so
that a sum over a row is off by at most ROW = 96 U of the sum of its terms' magnitudes, the terms' own roundings
included."""

from __future__ import annotations

import numpy as np

from tests.mx_util import f64, torch_dtype  # noqa: F401

U = 2.0 ** -24
ROW = 96 * U
HALF = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11, "float32": 2.0 ** -24}       # half a step, relative
TINY = {"bfloat16": 2.0 ** -134, "float16": 2.0 ** -25, "float32": 2.0 ** -150}    # half a subnormal step
DTYPES = ("bfloat16", "float16", "float32")


def rounded(value, before, dtype):
    """What a result may be off by: `before` its one rounding to dtype, and that rounding."""
    return before + HALF[dtype] * (np.abs(value) + before) + TINY[dtype]


def check(name, got, want, tol):
    bad = ~(np.abs(got - want) <= tol) & ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]} +- {np.broadcast_to(tol, got.shape)[bad][0]}")


def matrix(seed, rows, cols, dtype="bfloat16", std=1.0, ld=None, shift=0):
    """A seeded [rows, cols] tensor with outliers and a row of tiny values, `shift` elements into rows of `ld`, poison
    around them."""
    import torch
    rng = np.random.default_rng(seed)
    x = rng.normal(0, std, (rows, cols))
    x = np.where(rng.random(x.shape) < 0.01, x * 40, x)
    x[rows // 3] *= 2.0 ** -10
    t = torch.full((rows, (ld or cols) + shift), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    t[:, shift:shift + cols] = torch.from_numpy(x).to(torch_dtype(dtype))
    return t[:, shift:shift + cols]


def plan(seed, tokens, topk, groups, pad, drop=0.2):
    """The package's plan of random choices (distinct per token where there are enough experts), some of them dropped ->
    (row_off, src, pos) on the device and as numpy."""
    import torch

    import fp8_fine_grained_fp8bq_amd as fb
    rng = np.random.default_rng(seed)
    idx = np.argsort(rng.random((tokens, max(groups, topk))), 1)[:, :topk] % groups
    idx = np.where(rng.random(idx.shape) < drop, -1, idx).astype(np.int32)
    _, off, src, pos = fb.moe_plan(torch.from_numpy(idx).cuda(), groups, pad)
    return (off, src, pos), tuple(t.cpu().numpy() for t in (off, src, pos))
