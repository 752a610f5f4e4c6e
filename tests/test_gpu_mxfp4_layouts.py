"""Operands and outputs of the MXFP4 products on torch tensors whose strides are open or unusual (dimensions of one,
padded groups): the right values, or a refusal, and nothing outside the tensors touched."""

import numpy as np
import pytest

import fp8_fine_grained_fp8bq_amd as fb
from tests.gpu_util import log
from tests.mx_util import check_product, codes, f64, operand, torch_dtype

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups,k", [(2, 256), (5, 300), (17, 1057)])
@pytest.mark.parametrize("gap", [0, 16, 256])
def test_experts_of_one_row(groups, k, gap):
    """Codes [G, 1, bytes]: the stride of the dimension of one means nothing, the distance between groups does. The
    codes sit in a buffer of poison that also holds whatever that stride would lead to."""
    import torch
    log(f"experts of one row: {groups} groups, k {k}, gap {gap}")
    counts = np.arange(groups) % 4
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    m = int(off[-1]) + 1
    a, sa, va = operand(1, m, k)
    parts = [operand(10 + e, 1, k) for e in range(groups)]
    width = parts[0][0].shape[1]
    sb = torch.stack([p[1] for p in parts])
    for one in (width + gap, groups * (width + gap), 7 * 16, 3):         # strides of the dimension of one
        buf = torch.full((groups * groups * (width + gap),), 0x77, dtype=torch.uint8, device="cuda")
        b = buf.as_strided((groups, 1, width), (width + gap, one, 1))
        for e, p in enumerate(parts):
            b[e] = p[0]
        out = fb.grouped_gemm_mxfp4(torch.from_numpy(off).cuda(), a, sa, b, sb, dtype=torch.float32)
        got = f64(out)
        for e in range(groups):
            if counts[e]:
                check_product(got[off[e]:off[e + 1]], va[off[e]:off[e + 1]], parts[e][2], k, "float32")


def test_one_row_of_any_stride():
    """Dense operands of one row, whatever stride torch gives the row."""
    import torch
    k = 300
    a, sa, va = operand(1, 1, k)
    b, sb, vb = operand(2, 1, k)
    for stride in (1, 3, a.shape[1] + 5, 1 << 24):
        out = fb.gemm_mxfp4(a.as_strided(a.shape, (stride, 1)), sa, b.as_strided(b.shape, (stride, 1)), sb,
                            dtype=torch.float32)
        check_product(f64(out), va, vb, k, "float32")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n,gap", [(70, 0), (64, 8), (257, 3)])
def test_gradients_of_one_row(n, gap, dtype):
    """Experts' gradients [G, 1, n] in an output whose dimension of one has any stride: written at the distance between
    groups, nothing between them touched."""
    import torch
    groups = 3
    rng = np.random.default_rng(2)
    rows = 256 * groups
    off = torch.arange(0, rows + 1, 256, dtype=torch.int32, device="cuda")
    a, sa, _, _ = fb.quant_mxfp4_1x32(torch.from_numpy(rng.normal(size=(1, rows))).float().cuda())
    b, sb, _, _ = fb.quant_mxfp4_1x32(torch.from_numpy(rng.normal(size=(n, rows))).float().cuda())
    va, vb = codes(a, sa, rows), codes(b, sb, rows)
    for one in (n + gap, groups * (n + gap), 1, 5):
        buf = torch.full((groups * (n + gap),), 768.0, dtype=torch_dtype(dtype), device="cuda")
        out = buf.as_strided((groups, 1, n), (n + gap, one, 1))
        fb.grouped_wgrad_mxfp4(off, a, sa, b, sb, out=out)
        got = f64(out)
        for e in range(groups):
            part = slice(256 * e, 256 * e + 256)
            check_product(got[e], va[:, part], vb[:, part], 256, dtype)
        assert (buf.view(groups, n + gap)[:, n:] == 768.0).all()
    for strides in ((0, n, 1), (n - 1, n, 1)):
        with pytest.raises(ValueError, match="follow one another"):
            fb.grouped_wgrad_mxfp4(off, a, sa, b, sb, out=buf.as_strided((groups, 1, n), strides))
