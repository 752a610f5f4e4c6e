"""MXFP4 quantisation, dispatch and read-back on the GPU: codes and scales bit for bit those of the oracle."""

import numpy as np
import pytest

import fp8_fine_grained_fp8bq_amd as fb
from oracle import mxfp4
from tests.gpu_util import log
from tests.mx_util import DTYPES, f64, matrix, torch_dtype

pytestmark = pytest.mark.gpu


def same(q, s, want, what):
    wq, ws = want
    assert np.array_equal(s.cpu().numpy(), ws), f"{what}: scales differ"
    assert np.array_equal(q.cpu().numpy(), wq), f"{what}: codes differ"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("nosat", [False, True])
@pytest.mark.parametrize("rows,cols,ld", [(1, 1, 1), (1, 7168, 7168), (3, 33, 33), (17, 31, 40), (64, 256, 256),
                                          (130, 300, 301), (257, 513, 520), (300, 1057, 1057), (255, 64, 64)])
def test_both_forms(rows, cols, ld, dtype, nosat):
    log(f"quant {rows}x{cols} ld {ld} {dtype} nosat {nosat}")
    x = matrix(rows * 7 + cols, rows, cols, dtype, ld=ld)
    want = mxfp4.quantise(f64(x), nosat), mxfp4.quantise(f64(x).T, nosat)
    q, s, qt, st = fb.quant_mxfp4_1x32(x, colwise=True, nosat=nosat)
    same(q, s, want[0], "rows (both)")
    same(qt, st, want[1], "columns (both)")
    q, s, qt, st = fb.quant_mxfp4_1x32(x, nosat=nosat)
    assert qt is None and st is None
    same(q, s, want[0], "rows")
    q, s, qt, st = fb.quant_mxfp4_1x32(x, rowwise=False, colwise=True, nosat=nosat)
    assert q is None and s is None
    same(qt, st, want[1], "columns")


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_midpoint_and_its_neighbours(dtype):
    """Each tile: one element that fixes the scale, then the grid, its midpoints and the values next to them, under
    scales down to the smallest and up to the largest of the type."""
    import torch
    t = torch_dtype(dtype)
    fi = torch.finfo(t)
    base = torch.cat([torch.arange(0, 33, dtype=torch.float64) / 4, torch.tensor([0.1, 7.5, 7.9])])
    rows = []
    lo, hi = {"bfloat16": (-135, 125), "float16": (-24, 13), "float32": (-150, 125)}[dtype]
    for e in [lo, lo + 1, lo + 2, lo + 3, -128 if lo < -128 else lo + 5, -127 if lo < -127 else lo + 6, -126 if lo < -126 else lo + 7,
              -20, -1, 0, 1, hi - 1, hi]:
        v = (base * 2.0 ** e).to(t)
        up, dn = torch.nextafter(v, torch.full_like(v, float("inf"))), torch.nextafter(v, torch.zeros_like(v))
        v = torch.cat([v, up, dn, -v, -up, -dn])
        v = v[torch.isfinite(v)]
        top = torch.full((1,), min(7.9, 7.9) * 2.0 ** e if e < hi else float(fi.max), dtype=torch.float64).to(t)
        for i in range(0, len(v), 31):
            for m in (top, (torch.tensor([4.0 * 2.0 ** e], dtype=torch.float64)).to(t)):
                tile = torch.zeros(32, dtype=t)
                part = v[i:i + 31]
                tile[:len(part)] = part
                tile[31] = m
                rows.append(tile)
    x = torch.stack(rows)
    want = [mxfp4.quantise(f64(x), n) for n in (False, True)]
    for n in (False, True):
        q, s, _, _ = fb.quant_mxfp4_1x32(x.cuda(), nosat=n)
        same(q, s, want[n], f"midpoints nosat {n}")
        _, _, qt, st = fb.quant_mxfp4_1x32(x.t().contiguous().cuda(), rowwise=False, colwise=True, nosat=n)
        same(qt, st, want[n], f"midpoints, columns, nosat {n}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_nonfinite_tiles(dtype):
    import torch
    x = matrix(5, 70, 200, dtype)
    x[3, 5], x[40, 60], x[41, 199], x[69, 0] = float("nan"), float("inf"), -float("inf"), float("nan")
    q, s, qt, st = fb.quant_mxfp4_1x32(x, colwise=True)
    same(q, s, mxfp4.quantise(f64(x)), "rows")
    same(qt, st, mxfp4.quantise(f64(x).T), "columns")
    y = fb.dequant_mxfp4_1x32(q, s, 200, torch.float32)
    want = mxfp4.values(q.cpu().numpy(), s.cpu().numpy(), 200)
    assert np.array_equal(f64(y), want, equal_nan=True) and np.isnan(want).sum() > 100


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 255), (33, 256), (100, 1057)])
def test_read_back(rows, cols, dtype):
    x = matrix(11, rows, cols, "float32", std=0.1)
    q, s, _, _ = fb.quant_mxfp4_1x32(x)
    want = mxfp4.values(q.cpu().numpy(), s.cpu().numpy(), cols)
    y = fb.dequant_mxfp4_1x32(q, s, cols, torch_dtype(dtype))
    assert y.shape == (rows, cols) and y.dtype == torch_dtype(dtype)
    import torch
    rounded = torch.from_numpy(want).to(torch_dtype(dtype))     # exact but for fp16's range
    assert np.array_equal(f64(y), f64(rounded))


def test_read_back_of_every_code_and_scale():
    import torch
    q = torch.zeros((256, 128), dtype=torch.uint8)
    q[:, :16] = torch.arange(16, dtype=torch.uint8) * 16 + torch.arange(15, -1, -1, dtype=torch.uint8)
    s = torch.zeros((1, 256, 8), dtype=torch.uint8)
    s[0, :, 0] = torch.arange(256, dtype=torch.uint8)
    want = mxfp4.values(q.numpy(), s.numpy(), 32)
    y = fb.dequant_mxfp4_1x32(q.cuda(), s.cuda(), 32, torch.float32)
    with np.errstate(over="ignore"):
        assert np.array_equal(y.cpu().numpy(), want.astype(np.float32), equal_nan=True)
    y = fb.dequant_mxfp4_1x32(q.cuda(), s.cuda(), 32)
    assert np.array_equal(f64(y)[:252], want[:252], equal_nan=True)      # below bf16's overflow


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("xrows,cols,rows", [(1, 40, 5), (50, 300, 257), (64, 512, 300)])
def test_dispatch(xrows, cols, rows, dtype):
    """Rows by index: repeated, missing (-1) and out-of-range entries, which give zero rows."""
    import torch
    x = matrix(21, xrows, cols, dtype)
    rng = np.random.default_rng(3)
    src = rng.integers(0, xrows, rows).astype(np.int32)
    src[rng.random(rows) < 0.2] = -1
    src[0], src[-1] = xrows, -(1 << 31)
    xs = np.where(((src >= 0) & (src < xrows))[:, None], f64(x)[np.clip(src, 0, xrows - 1)], 0.0)
    q, s, qt, st = fb.dispatch_mxfp4_1x32(x, torch.from_numpy(src).cuda(), colwise=True)
    same(q, s, mxfp4.quantise(xs), "rows")
    same(qt, st, mxfp4.quantise(xs.T), "columns")
    q, s, _, _ = fb.dispatch_mxfp4_1x32(x, torch.from_numpy(src).cuda())
    same(q, s, mxfp4.quantise(xs), "rows only")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("nosat", [False, True])
@pytest.mark.parametrize("xrows,cols,rows", [(1, 40, 2), (1, 7168, 300), (50, 300, 257), (33, 513, 1000)])
def test_dispatch_with_a_workspace(xrows, cols, rows, dtype, nosat):
    """Each source row read once (rows >= 2 xrows), also where more rows show it than it has slots: the same codes;
    unused rows keep their bytes, twice over."""
    import torch
    x = matrix(23, xrows, cols, dtype)
    rng = np.random.default_rng(4)
    src = rng.integers(-2, xrows + 2, rows).astype(np.int32)
    xs = np.where(((src >= 0) & (src < xrows))[:, None], f64(x)[np.clip(src, 0, xrows - 1)], 0.0)
    wq, ws = mxfp4.quantise(xs, nosat)
    unused = src == -2
    chunks = ws.shape[0]
    d = torch.from_numpy(src).cuda()
    work = torch.full((xrows * fb.DISPATCH_WORKSPACE_ROW_BYTES // 4 + 1,), 77, dtype=torch.int32, device="cuda")
    for _ in range(2):
        q = torch.full((rows, chunks * 128 + 16), 0xAB, dtype=torch.uint8, device="cuda")
        s = torch.full((chunks, rows + 1, 8), 0xCD, dtype=torch.uint8, device="cuda")
        fb.fp8bq_dispatch_mxfp4_1x32(x.data_ptr(), fb.BF16 if dtype == "bfloat16" else fb.FP16 if dtype == "float16" else fb.FP32,
                                     xrows, cols, cols, d.data_ptr(), rows, q.data_ptr(), q.shape[1], s.data_ptr(), rows + 1,
                                     None, 0, None, 0, fb.MX_NOSAT if nosat else 0, work.data_ptr(),
                                     torch.cuda.current_stream().cuda_stream)
        gq, gs = q.cpu().numpy(), s.cpu().numpy()
        assert np.array_equal(gq[~unused, :chunks * 128], wq[~unused]) and np.array_equal(gs[:, :rows][:, ~unused], ws[:, ~unused])
        assert (gq[unused] == 0xAB).all() and (gq[:, chunks * 128:] == 0xAB).all()
        assert (gs[:, rows] == 0xCD).all() and (gs[:, :rows][:, unused] == 0xCD).all()
        assert int(work[-1]) == 77


def test_dispatch_leaves_unused_rows():
    """Rows marked unused keep their bytes in the row form and are zeros in the column form."""
    import torch
    x = matrix(22, 30, 300)
    src = torch.tensor([3, -2, 29, -1, -2, -2], dtype=torch.int32, device="cuda")
    xs = np.zeros((6, 300))
    xs[0], xs[2] = f64(x)[3], f64(x)[29]
    wq, ws = mxfp4.quantise(xs)
    for both in (False, True):
        q = torch.full((6, 256), 0xAB, dtype=torch.uint8, device="cuda")
        s = torch.full((2, 6, 8), 0xCD, dtype=torch.uint8, device="cuda")
        qt = torch.empty((300, 128), dtype=torch.uint8, device="cuda")
        st = torch.empty((1, 300, 8), dtype=torch.uint8, device="cuda")
        fb.fp8bq_dispatch_mxfp4_1x32(x.data_ptr(), fb.BF16, 30, 300, 300, src.data_ptr(), 6, q.data_ptr(), 256,
                                     s.data_ptr(), 6, *((qt.data_ptr(), 128, st.data_ptr(), 300) if both else (None, 0, None, 0)),
                                     0, None, torch.cuda.current_stream().cuda_stream)
        used = [0, 2, 3]
        assert np.array_equal(q[used].cpu().numpy(), wq[used]) and np.array_equal(s[:, used].cpu().numpy(), ws[:, used])
        assert (q[[1, 4, 5]] == 0xAB).all() and (s[:, [1, 4, 5]] == 0xCD).all()
    same(qt, st, mxfp4.quantise(xs.T), "columns")


def test_outputs_stay_inside_their_buffers():
    """Larger leading dimensions through the C entry: nothing between the rows or behind the last is written."""
    import torch
    rows, cols = 70, 300
    x = matrix(9, rows, cols)
    q = torch.full((rows + 1, 512), 0xAB, dtype=torch.uint8, device="cuda")
    s = torch.full((2, rows + 3, 8), 0xCD, dtype=torch.uint8, device="cuda")
    qt = torch.full((cols + 1, 160), 0xAB, dtype=torch.uint8, device="cuda")
    st = torch.full((1, cols + 5, 8), 0xCD, dtype=torch.uint8, device="cuda")
    fb.fp8bq_quant_mxfp4_1x32(x.data_ptr(), fb.BF16, rows, cols, x.stride(0), q.data_ptr(), 512, s.data_ptr(), rows + 3,
                              qt.data_ptr(), 160, st.data_ptr(), cols + 5, 0, torch.cuda.current_stream().cuda_stream)
    want, wantt = mxfp4.quantise(f64(x)), mxfp4.quantise(f64(x).T)
    assert np.array_equal(q[:rows, :256].cpu().numpy(), want[0]) and np.array_equal(s[:, :rows].cpu().numpy(), want[1])
    assert np.array_equal(qt[:cols, :128].cpu().numpy(), wantt[0]) and np.array_equal(st[:, :cols].cpu().numpy(), wantt[1])
    assert (q[:, 256:] == 0xAB).all() and (q[rows:] == 0xAB).all() and (s[:, rows:] == 0xCD).all()
    assert (qt[:, 128:] == 0xAB).all() and (qt[cols:] == 0xAB).all() and (st[:, cols:] == 0xCD).all()


def test_more_than_2_31_elements():
    """Rows behind 2^31 elements (and 4 GiB) in both forms: the same bytes as those of the last rows alone."""
    import torch
    rows, cols = 300_032, 7168
    log(f"quant {rows}x{cols}")
    x = torch.randn((rows // 64, cols), dtype=torch.bfloat16, device="cuda").repeat(64, 1)
    q, s, qt, st = fb.quant_mxfp4_1x32(x, colwise=True)
    last = 512
    lq, ls, lqt, lst = fb.quant_mxfp4_1x32(x[-last:].contiguous(), colwise=True)
    assert (q[-last:] == lq).all() and (s[:, -last:] == ls).all()
    assert (qt[:, -last // 2:] == lqt).all() and (st[-last // 256:] == lst).all()
    y = fb.dequant_mxfp4_1x32(q, s, cols)
    assert (y[-last:] == fb.dequant_mxfp4_1x32(lq, ls, cols)).all()
