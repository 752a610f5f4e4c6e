"""MXFP4 products on the GPU against float64: dense, rows grouped by expert, weight gradients of experts."""

import numpy as np
import pytest

import fp8_fine_grained_fp8bq_amd as fb
from tests.gpu_util import log
from tests.mx_util import check_product, codes, f64, matrix, operand, torch_dtype

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 1), (1, 2048, 1024), (2, 33, 96), (31, 64, 256), (32, 32, 32), (33, 257, 1057), (48, 520, 2048),
         (100, 1001, 300), (128, 128, 512), (129, 384, 513), (256, 256, 256), (257, 1000, 768), (300, 515, 1536),
         (512, 768, 1024), (700, 260, 2080)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_dense(m, n, k, dtype):
    log(f"gemm_mxfp4 {m}x{n}x{k} {dtype}")
    a, sa, va = operand(m + 1, m, k)
    b, sb, vb = operand(n + 2, n, k)
    out = fb.gemm_mxfp4(a, sa, b, sb, dtype=torch_dtype(dtype))
    assert out.shape == (m, n)
    check_product(f64(out), va, vb, k, dtype)
    again = fb.gemm_mxfp4(a, sa, b, sb, dtype=torch_dtype(dtype))
    assert (out == again).all(), "not the same at every call"


@pytest.mark.parametrize("m,n,k", [(4096, 2048, 7168), (1500, 4096, 2048), (2048, 7168, 4096), (64, 7168, 2048),
                                   (200, 18432, 1024)])
def test_dense_large(m, n, k):
    """The larger tilings, against a float64 product on the GPU of the decoded values."""
    import torch
    log(f"gemm_mxfp4 {m}x{n}x{k}")
    x, w = matrix(1, m, k), matrix(2, n, k, std=0.02)
    a, sa, _, _ = fb.quant_mxfp4_1x32(x)
    b, sb, _, _ = fb.quant_mxfp4_1x32(w)
    va = fb.dequant_mxfp4_1x32(a, sa, k, torch.float32).double()
    vb = fb.dequant_mxfp4_1x32(b, sb, k, torch.float32).double().t().contiguous()
    exact, ab = va @ vb, va.abs() @ vb.abs()
    tol = (k + 64) * 2.0 ** -23 * ab
    out = fb.gemm_mxfp4(a, sa, b, sb, dtype=torch.float32)
    assert ((out.double() - exact).abs() <= tol).all()
    out = fb.gemm_mxfp4(a, sa, b, sb)
    assert ((out.double() - exact).abs() <= tol + 2.0 ** -8 * (exact.abs() + tol)).all()


@pytest.mark.parametrize("m,n,k", [(3, 40, 64), (70, 300, 600), (260, 512, 512)])
def test_output_views_and_poison(m, n, k):
    """A view with a longer, unaligned row stride: only its own elements are written."""
    import torch
    a, sa, va = operand(1, m, k)
    b, sb, vb = operand(2, n, k)
    for dtype in ("bfloat16", "float32"):
        for off, ld in ((0, n + 8), (1, n + 3)):
            buf = torch.full((m + 2, ld), 768.0, dtype=torch_dtype(dtype), device="cuda")
            out = buf[:m, off:off + n]
            fb.gemm_mxfp4(a, sa, b, sb, out=out)
            check_product(f64(out), va, vb, k, dtype)
            buf[:m, off:off + n] = 768.0
            assert (buf == 768.0).all()


def test_padded_operands():
    """Codes and scales as views of larger buffers whose other bytes are poison."""
    import torch
    m, n, k = 65, 70, 520
    a, sa, va = operand(1, m, k)
    b, sb, vb = operand(2, n, k)
    bufs = []
    for q, s in ((a, sa), (b, sb)):
        qq = torch.full((q.shape[0] + 1, q.shape[1] + 32), 0x77, dtype=torch.uint8, device="cuda")
        ss = torch.full((s.shape[0], s.shape[1] + 3, 8), 0xFF, dtype=torch.uint8, device="cuda")
        qq[:-1, :q.shape[1]], ss[:, :s.shape[1]] = q, s
        bufs += [qq[:-1, :q.shape[1]], ss[:, :s.shape[1]]]
    check_product(f64(fb.gemm_mxfp4(*bufs)), va, vb, k, "bfloat16")


def test_nan_tiles_reach_their_rows_and_columns_only():
    import torch
    m, n, k = 40, 300, 512
    x, w = matrix(3, m, k), matrix(4, n, k)
    x[7, 100], w[33, 500] = float("nan"), float("inf")
    a, sa, _, _ = fb.quant_mxfp4_1x32(x)
    b, sb, _, _ = fb.quant_mxfp4_1x32(w)
    for big in (False, True):
        if big:     # the same rows in the middle of a product of many rows
            a, sa, _, _ = fb.quant_mxfp4_1x32(torch.cat([matrix(5, 600, k), x]))
        out = f64(fb.gemm_mxfp4(a, sa, b, sb))[-m:]
        nan = np.isnan(out)
        assert nan[7].all() and nan[:, 33].all() and nan.sum() == m + n - 1


@pytest.mark.parametrize("scale", [-60, 60])
def test_extreme_scales(scale):
    """Scale bytes far from one: products that stay inside fp32 keep their accuracy."""
    import torch
    a, sa, va = operand(1, 40, 300)
    b, sb, vb = operand(2, 50, 300)
    sa2 = torch.where(sa > 0, sa + scale, sa) if scale > 0 else torch.where(sa > 60, sa - 60, sa)
    out = fb.gemm_mxfp4(a, sa2, b, sb, dtype=torch.float32)
    check_product(f64(out) * 2.0 ** -scale, va, vb, 300, "float32")


def offsets(counts, pad=1):
    off = [0]
    for c in counts:
        off.append(off[-1] + -(-c // pad) * pad)
    return np.array(off, np.int32)


COUNTS = [[5], [0, 0, 3], [1, 0, 40, 2], [33, 64, 0, 0, 129], [300, 1, 31, 0, 32, 257], [0, 0], [1] * 70,
          [0] * 200 + [7] + [0] * 55, [600, 5], [3] * 256]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_grouped_rows(counts, dtype):
    import torch
    g = len(counts)
    n, k = (40, 96) if g > 60 else (300, 600)
    off = offsets(counts)
    spare = 5
    m = int(off[-1]) + spare
    log(f"grouped {counts[:8]} n {n} k {k}")
    a, sa, va = operand(1, m, k)
    parts = [operand(10 + e, n, k) for e in range(g)]
    b, sb = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    out = torch.full((m, n), 768.0, dtype=torch_dtype(dtype), device="cuda")
    fb.grouped_gemm_mxfp4(torch.from_numpy(off).cuda(), a, sa, b, sb, out=out)
    got = f64(out)
    for e in range(g):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            check_product(got[lo:hi], va[lo:hi], parts[e][2], k, dtype)
    assert (got[off[-1]:] == 768.0).all(), "rows behind the last expert were written"


@pytest.mark.parametrize("rows", [[700, 0, 1300, 513], [2, 9, 4, 1, 0, 30, 17, 8], [60, 100, 250, 31]])
def test_grouped_rows_large(rows):
    """Wide weights, few and many rows per expert, against the dense product of each expert's rows."""
    import torch
    off = offsets(rows)
    m, n, k = int(off[-1]), 2048, 1536
    x, w = matrix(1, m, k), matrix(2, len(rows) * n, k, std=0.02)
    a, sa, _, _ = fb.quant_mxfp4_1x32(x)
    qs = [fb.quant_mxfp4_1x32(v)[:2] for v in w.view(len(rows), n, k)]
    out = fb.grouped_gemm_mxfp4(torch.from_numpy(off).cuda(), a, sa, torch.stack([q for q, _ in qs]),
                                torch.stack([s for _, s in qs]), dtype=torch.float32)
    va = fb.dequant_mxfp4_1x32(a, sa, k, torch.float32).double()
    for e, (q, s) in enumerate(qs):
        vb = fb.dequant_mxfp4_1x32(q, s, k, torch.float32).double().t().contiguous()
        va_e = va[off[e]:off[e + 1]]
        tol = (k + 64) * 2.0 ** -23 * (va_e.abs() @ vb.abs())
        assert ((out[off[e]:off[e + 1]].double() - va_e @ vb).abs() <= tol).all(), f"expert {e}"


def test_broken_offsets_stay_inside():
    """Offsets outside [0, m] and decreasing ones are clamped: in-range groups are right, nothing outside is touched."""
    import torch
    m, n, k = 50, 64, 64
    a, sa, va = operand(1, m, k)
    b, sb, vb = operand(2, n, k)
    out = torch.full((m + 4, n), 768.0, dtype=torch.float32, device="cuda")
    off = torch.tensor([-5, 20, 10, 1 << 30], dtype=torch.int32, device="cuda")
    fb.grouped_gemm_mxfp4(off, a, sa, b.expand(3, *b.shape).contiguous(), sb.expand(3, *sb.shape).contiguous(), out=out[:m])
    check_product(f64(out[:m]), va, vb, k, "float32")
    assert (out[m:] == 768.0).all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("counts", [[256], [0, 300, 1, 0, 512], [257] * 3 + [0], [1] * 12], ids=str)
@pytest.mark.parametrize("m,n", [(40, 70), (300, 129)])
def test_grouped_wgrad(counts, m, n, dtype):
    import torch
    off = offsets(counts, 256)
    rows = int(off[-1]) + 256                      # a chunk of rows behind the last expert
    rng = np.random.default_rng(5)
    dy, x = rng.normal(size=(rows, m)), rng.normal(size=(rows, n))
    for e, c in enumerate(counts):
        dy[off[e] + c:off[e + 1]] = 0
    a, sa, _, _ = fb.quant_mxfp4_1x32(torch.from_numpy(dy.T.copy()).float().cuda())
    b, sb, _, _ = fb.quant_mxfp4_1x32(torch.from_numpy(x.T.copy()).float().cuda())
    out = torch.full((len(counts), m, n), 768.0, dtype=torch_dtype(dtype), device="cuda")
    fb.grouped_wgrad_mxfp4(torch.from_numpy(off).cuda(), a, sa, b, sb, out=out)
    va, vb, got = codes(a, sa, rows), codes(b, sb, rows), f64(out)
    for e in range(len(counts)):
        lo, hi = off[e], off[e + 1]
        check_product(got[e], va[:, lo:hi], vb[:, lo:hi], hi - lo, dtype)
        if counts[e] == 0:
            assert (got[e] == 0).all()


@pytest.mark.parametrize("m,n,k", [(70, 90, 110), (256, 320, 288)])
def test_linear_training_step(m, n, k):
    """Forward, gradient of the input and of the weight of y = x w^T, each the product of the quantised operands."""
    import torch
    x, w, dy = matrix(1, m, k), matrix(2, n, k, std=0.02), matrix(3, m, n, std=1e-3)
    xq, xs, xqt, xst = fb.quant_mxfp4_1x32(x, colwise=True)
    wq, ws, wqt, wst = fb.quant_mxfp4_1x32(w, colwise=True)
    gq, gs, gqt, gst = fb.quant_mxfp4_1x32(dy, colwise=True)
    check_product(f64(fb.gemm_mxfp4(xq, xs, wq, ws)), codes(xq, xs, k), codes(wq, ws, k), k, "bfloat16")
    check_product(f64(fb.gemm_mxfp4(gq, gs, wqt, wst)), codes(gq, gs, n), codes(wqt, wst, n), n, "bfloat16")
    check_product(f64(fb.gemm_mxfp4(gqt, gst, xqt, xst, dtype=torch.float32)), codes(gqt, gst, m), codes(xqt, xst, m),
                  m, "float32")


def test_other_stream_and_graph_replays():
    """On a side stream, and captured: every replay sees the buffers' present contents."""
    import torch
    m, n, k = 300, 520, 700
    x, w = matrix(1, m, k), matrix(2, n, k)
    wq, ws, _, _ = fb.quant_mxfp4_1x32(w)

    def step(v):
        q, s, _, _ = fb.quant_mxfp4_1x32(v)
        return fb.gemm_mxfp4(q, s, wq, ws)

    want = step(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(x)
    side.synchronize()
    assert (got == want).all()
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(buf)
    for seed in (7, 8, 9):
        new = matrix(seed, m, k)
        buf.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert (out == step(new)).all()


def _raw(rows, chunks, seed):
    """Random codes and scales made on the device."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    q = torch.randint(0, 256, (rows, chunks * 128), dtype=torch.uint8, device="cuda", generator=gen)
    s = torch.randint(120, 130, (chunks, rows, 8), dtype=torch.uint8, device="cuda", generator=gen)
    return q, s


@pytest.mark.parametrize("m,n,chunks", [(2_200_000, 8, 1), (34_000_000, 5, 1), (70_000, 40, 260)])
def test_tall_products(m, n, chunks):
    """Many tiles of few columns; operands and offsets past 2 and 4 GiB: rows at both ends and around the powers of two
    against the product of those rows alone."""
    import torch
    log(f"tall product {m}x{n}, {chunks} chunks")
    a, sa = _raw(m, chunks, 1)
    b, sb = _raw(n, chunks, 2)
    out = fb.gemm_mxfp4(a, sa, b, sb, dtype=torch.float32)
    k = chunks * 256
    vb = codes(b, sb, k)
    for at in sorted({0, m // 3, m - 64, min(m - 64, (1 << 24) - 32), min(m - 64, (1 << 25) - 32)}):
        va = codes(a[at:at + 64], sa[:, at:at + 64].contiguous(), k)
        check_product(f64(out[at:at + 64]), va, vb, k, "float32")


def test_wide_product():
    """A weight of millions of rows against one token."""
    import torch
    m, n, chunks = 1, 3_000_000, 1
    a, sa = _raw(m, chunks, 3)
    b, sb = _raw(n, chunks, 4)
    out = fb.gemm_mxfp4(a, sa, b, sb)
    va = codes(a, sa, 256)
    for at in (0, n // 2 + 7, n - 64):
        vb = codes(b[at:at + 64], sb[:, at:at + 64].contiguous(), 256)
        check_product(f64(out[:, at:at + 64]), va, vb, 256, "bfloat16")
