"""The upper end of MXFP4's range: what saturates, and what the scales that never saturate round past fp32."""

import pytest

import fp8_fine_grained_fp8bq_amd as fb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("factor,plain,nosat", [(1.0, 1.0, 1.0), (1.70, 1.5, 1.5), (1.90, 1.5, float("inf"))])
def test_largest_magnitudes(factor, plain, nosat):
    import torch
    top = 2.0 ** 127
    x = torch.zeros((2, 64))
    x[0, 3], x[1, 40] = factor * top, -factor * top
    one = torch.zeros((1, 64), device="cuda")
    one[0, 3] = 1.0
    qb, sb, _, _ = fb.quant_mxfp4_1x32(one)
    for flag, want in ((False, plain), (True, nosat)):
        q, s, _, _ = fb.quant_mxfp4_1x32(x.cuda(), nosat=flag)
        for dtype in (torch.float32, torch.bfloat16):
            y = fb.dequant_mxfp4_1x32(q, s, 64, dtype)
            assert float(y[0, 3]) == want * top and float(y[1, 40]) == -want * top
        assert float(fb.gemm_mxfp4(q, s, qb, sb, dtype=torch.float32)[0, 0]) == want * top
