"""Layouts that the tensor layer refuses before it looks at the device. Runs without a GPU."""

import pytest

import fp8_fine_grained_fp8bq_amd as fb


@pytest.mark.parametrize("rows,strides", [(1, (0, 128, 1)), (1, (64, 128, 1)), (1, (112, 3, 1)), (2, (384, 128, 1)),
                                          (2, (256, 0, 1)), (2, (128, 64, 1))])
def test_groups_that_do_not_follow_one_another(rows, strides):
    import torch
    a, sa = torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((1, 4, 8), dtype=torch.uint8)
    off = torch.zeros(4, dtype=torch.int32)
    b = torch.zeros(4096, dtype=torch.uint8).as_strided((3, rows, 128), strides)
    with pytest.raises(ValueError, match="follow one another"):
        fb.grouped_gemm_mxfp4(off, a, sa, b, torch.zeros((3, 1, rows, 8), dtype=torch.uint8))


@pytest.mark.parametrize("strides", [(128, 384, 1), (128, 1, 1), (256, 3, 1)])
def test_stride_of_a_single_row_is_open(strides):
    """Groups of one row: only the distance between groups counts; such codes get as far as the device check."""
    import torch
    a, sa = torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((1, 4, 8), dtype=torch.uint8)
    off = torch.zeros(4, dtype=torch.int32)
    b = torch.zeros(4096, dtype=torch.uint8).as_strided((3, 1, 128), strides)
    with pytest.raises(ValueError, match="must be on the GPU"):
        fb.grouped_gemm_mxfp4(off, a, sa, b, torch.zeros((3, 1, 1, 8), dtype=torch.uint8))
