"""Every tiling of the MXFP4 products, dense, over experts' rows and for experts' weight gradients, at the sizes of
tests/mx_tilings.py, against float64 products (on the GPU) of the values that the operands stand for: both output types,
rows of any stride with poison around them, operands inside larger buffers, NaN tiles, experts without rows."""

import pytest

import fp8_fine_grained_fp8bq_amd as fb
from tests import mx_tilings as mt
from tests.gpu_util import log
from tests.mx_util import matrix, torch_dtype

pytestmark = pytest.mark.gpu

POISON = 768.0
IDS = dict(ids=lambda v: str(v)[:24])


def operand(seed, rows, k, std=1.0):
    """Codes and scales of a random matrix, and their values (float64, on the GPU)."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, k), generator=gen, device="cuda") * std
    x *= torch.exp2(torch.randint(-3, 4, (rows, 1), generator=gen, device="cuda").float())
    q, s, _, _ = fb.quant_mxfp4_1x32(x)
    return q, s, fb.dequant_mxfp4_1x32(q, s, k, torch.float32).double()


def check(out, va, vb, k, dtype):
    """out [m, n] against va vb^T: at most k fp32 additions, each off by at most 2^-23 of sum |a||b|, and bf16's half
    step."""
    bt = vb.t().contiguous()
    exact = va @ bt
    tol = (k + 64) * 2.0 ** -23 * (va.abs() @ bt.abs())
    if dtype == "bfloat16":
        tol = tol + 2.0 ** -8 * (exact.abs() + tol) + 2.0 ** -134
    bad = ~((out.double() - exact).abs() <= tol)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"


def inside(q, s):
    """The same operand inside larger buffers of poison."""
    import torch
    qq = torch.full((q.shape[0] + 1, q.shape[1] + 48), 0x77, dtype=torch.uint8, device="cuda")
    ss = torch.full((s.shape[0], s.shape[1] + 3, 8), 0xFF, dtype=torch.uint8, device="cuda")
    qq[:-1, :q.shape[1]], ss[:, :s.shape[1]] = q, s
    return qq[:-1, :q.shape[1]], ss[:, :s.shape[1]]


def output(shape, dtype, odd):
    """An output of poison, rows aligned or not, with poison around it: (buffer, view)."""
    import torch
    lead, gap = (1, 3) if odd else (0, -shape[-1] % 8)
    buf = torch.full((*shape[:-1], lead + shape[-1] + gap), POISON, dtype=torch_dtype(dtype), device="cuda")
    return buf, buf[..., lead:lead + shape[-1]]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("tiling,several,m,n,k", mt.DENSE, **IDS)
def test_dense(tiling, several, m, n, k, dtype):
    log(f"dense {tiling} {m}x{n}x{k} {dtype}")
    a, sa, va = operand(1, m, k)
    b, sb, vb = operand(2, n, k, 0.02)
    first = None
    for odd in (False, True):
        buf, out = output((m, n), dtype, odd)
        fb.gemm_mxfp4(*(inside(a, sa) if odd else (a, sa)), *(inside(b, sb) if odd else (b, sb)), out=out)
        check(out, va, vb, k, dtype)
        if first is not None:
            assert (out == first).all(), "another row stride, another result"
        first = out.clone()
        out.fill_(POISON)
        assert (buf == POISON).all(), "written outside the output"


@pytest.mark.parametrize("tiling,several,m,n,k", mt.DENSE, **IDS)
def test_nan_tiles_reach_their_rows_and_columns_only(tiling, several, m, n, k):
    import torch
    log(f"NaN {tiling} {m}x{n}x{k}")
    x, w = matrix(3, m, k), matrix(4, n, k)
    row, col = m - 2, n // 2
    x[row, k - 1], w[col, 100] = float("nan"), float("inf")
    out = fb.gemm_mxfp4(*fb.quant_mxfp4_1x32(x)[:2], *fb.quant_mxfp4_1x32(w)[:2])
    nan = torch.isnan(out)
    assert bool(nan[row].all()) and bool(nan[:, col].all()) and int(nan.sum()) == m + n - 1


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("tiling,several,m,n,k,counts", mt.ROWS, **IDS)
def test_rows(tiling, several, m, n, k, counts, dtype):
    import torch
    log(f"rows {tiling} {m}x{n}x{k} of {counts} {dtype}")
    g, off = len(counts), mt.padded(counts, 1)
    a, sa, va = operand(1, m, k)
    parts = [operand(10 + e, n, k, 0.02) for e in range(g)]
    b, sb = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    doff = torch.tensor(off, dtype=torch.int32, device="cuda")
    for odd in (False, True):
        buf, out = output((m, n), dtype, odd)
        fb.grouped_gemm_mxfp4(doff, *(inside(a, sa) if odd else (a, sa)), b, sb, out=out)
        for e in range(g):
            if counts[e]:
                check(out[off[e]:off[e + 1]], va[off[e]:off[e + 1]], parts[e][2], k, dtype)
        out[:off[-1]].fill_(POISON)
        assert (buf == POISON).all(), "written outside the experts' rows"


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("tiling,several,m,n,counts", mt.WGRAD, **IDS)
def test_weight_gradients(tiling, several, m, n, counts, dtype):
    import torch
    log(f"wgrad {tiling} {m}x{n} of {counts} {dtype}")
    g, off = len(counts), mt.padded(counts, 256)
    rows = off[-1] + 256                              # a chunk of rows behind the last expert, of any content
    gen = torch.Generator(device="cuda").manual_seed(5)
    dy, x = torch.randn((rows, m), generator=gen, device="cuda"), torch.randn((rows, n), generator=gen, device="cuda")
    for e, c in enumerate(counts):
        dy[off[e] + c:off[e + 1]] = 0
        x[off[e] + c:off[e + 1]] = 0
    dy[off[-1]:] = float("nan")
    _, _, a, sa = fb.quant_mxfp4_1x32(dy, rowwise=False, colwise=True)
    _, _, b, sb = fb.quant_mxfp4_1x32(x, rowwise=False, colwise=True)
    va, vb = (fb.dequant_mxfp4_1x32(q, s, rows, torch.float32).double() for q, s in ((a, sa), (b, sb)))
    doff = torch.tensor(off, dtype=torch.int32, device="cuda")
    for odd in (False, True):
        buf, out = output((g, m, n), dtype, odd)
        fb.grouped_wgrad_mxfp4(doff, *(inside(a, sa) if odd else (a, sa)), *(inside(b, sb) if odd else (b, sb)), out=out)
        for e in range(g):
            lo, hi = off[e], off[e + 1]
            if counts[e]:
                check(out[e], va[:, lo:hi], vb[:, lo:hi], hi - lo, dtype)
            else:
                assert (out[e] == 0).all(), f"expert {e} has no rows"
        out.fill_(POISON)
        assert (buf == POISON).all(), "written outside the gradients"


@pytest.mark.parametrize("which", ["first", "last", "all"])
@pytest.mark.parametrize("tiling,m,n", mt.WGRAD_FEW)
def test_weight_gradients_of_few_experts(tiling, m, n, which):
    """Only the first, only the last, or no expert has rows: the others' gradients are zeros."""
    import torch
    counts = {"first": [600, 0, 0, 0], "last": [0, 0, 0, 600], "all": [0, 0, 0, 0]}[which]
    log(f"wgrad {tiling} {m}x{n} of {counts}")
    off, rows = mt.padded(counts, 256), 1024
    a, sa, va = operand(1, m, rows)
    b, sb, vb = operand(2, n, rows)
    out = fb.grouped_wgrad_mxfp4(torch.tensor(off, dtype=torch.int32, device="cuda"), a, sa, b, sb)
    for e, c in enumerate(counts):
        if c:
            check(out[e], va[:, off[e]:off[e + 1]], vb[:, off[e]:off[e + 1]], 768, "float32")
        else:
            assert (out[e] == 0).all()
