"""Sizes at the limit of the MXFP4 quantisers' grids: what a launch could not hold (2^32 threads) is refused as too
large, and nothing smaller. Runs without a GPU."""

import os

import pytest

import fp8_fine_grained_fp8bq_amd as fb

A16, S8, O4 = 0x10000, 0x20008, 0x30004       # never dereferenced
LIMIT = 1 << 24                               # blocks of 256 threads


def row_blocks(rows, cols):
    return -(-rows // 16) * -(-cols // 256)   # an upper bound: a block takes 16 rows of a pair of chunks


def column_blocks(rows, cols, size):
    return -(-rows // 256) * -(-cols // 256) * (2 * 256 // (128 // size))


CASES = [(16768, 4_096_000), (16384, 4_096_000), (16385, 4_096_000), (16512, 4_079_000), (257, 4_194_048), (1, 4_194_048),
         (16_000_000, 4096), (16_777_216, 4096), (16_384, 4_194_048), (16_640, 4_144_000)]


@pytest.mark.parametrize("rows,cols", CASES)
@pytest.mark.parametrize("xtype,size", [(fb.BF16, 2), (fb.FP16, 2), (fb.FP32, 4)])
@pytest.mark.parametrize("form", ["rows", "columns", "both"])
@pytest.mark.parametrize("indexed", [False, True])
def test_grid_limits(rows, cols, xtype, size, form, indexed):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible; valid arguments would launch")
    if not os.path.exists(fb.LIB_PATH):
        pytest.skip("libfp8bq.so not built (run __graft_entry__.build())")
    ldq, ldqt = -(-cols // 256) * 128, -(-rows // 256) * 128
    out = [A16, ldq, S8, rows] if form != "columns" else [None, 0, None, 0]
    out += [A16, ldqt, S8, cols] if form != "rows" else [None, 0, None, 0]
    if indexed:
        status = fb.lib().fp8bq_dispatch_mxfp4_1x32(A16, xtype, 40, cols, cols, O4, rows, *out, 0, None, None)
    else:
        status = fb.lib().fp8bq_quant_mxfp4_1x32(A16, xtype, rows, cols, cols, *out, 0, None)
    fits = row_blocks(rows, cols) < LIMIT
    if form != "rows":
        fits = fits and ldqt < 1 << 23 and column_blocks(rows, cols, size) < LIMIT
    assert status == (fb.E_DEVICE if fits else fb.E_SHAPE), fb.lib().fp8bq_last_error()
