"""Products of unquantised rows with MXFP4 weights, dense and over experts, against float64: row counts from one to several
tiles, odd sizes, types, strides, scales at the ends of their range."""

import numpy as np
import pytest

import fp8_fine_grained_fp8bq_amd as fb
from oracle import mxfp4
from tests.gpu_util import log
from tests.layer_util import DTYPES, check, f64, matrix, rounded, torch_dtype
from tests.mx_util import accumulation_bound, operand

pytestmark = pytest.mark.gpu


def check_product(out, vx, vw, k, xtype, otype):
    """x is split into up to three terms, each with k products."""
    terms = {"bfloat16": 1, "float16": 2, "float32": 3}[xtype]
    want = vx @ vw.T
    check("out", out, want, rounded(want, accumulation_bound(terms * k, np.abs(vx) @ np.abs(vw).T), otype))


@pytest.mark.parametrize("xtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 16, 32), (1, 17, 31), (1, 2048, 7168), (2, 33, 33), (3, 64, 255), (7, 100, 256),
                                   (15, 48, 257), (16, 64, 512), (17, 50, 700), (31, 129, 1057), (32, 32, 2048), (48, 16, 96),
                                   (64, 80, 640), (65, 96, 1000), (130, 40, 300), (5, 18432, 128),
                                   (12, 4100, 520), (20, 4097, 300), (12, 12301, 300), (16, 12288, 1030), (4, 8003, 300),
                                   (3, 9001, 300), (4, 13001, 300), (3, 17003, 1300), (8, 8003, 300), (5, 9001, 300), (7, 13001, 520),
                                   (6, 17003, 300), (9, 8003, 300), (13, 9001, 520), (12, 13001, 300), (14, 17003, 300), (33, 6001, 300)])
def test_product(m, n, k, xtype):
    log(f"gemv {m}x{n}x{k} {xtype}")
    w, ws, vw = operand(n + k, n, k)
    for shift in (0, 1):
        x = matrix(m, m, k, xtype, ld=k + 3 * shift, shift=shift)
        check_product(f64(fb.gemv_mxfp4(x, w, ws)), f64(x), vw, k, xtype, xtype)
    for otype in DTYPES:
        check_product(f64(fb.gemv_mxfp4(x, w, ws, dtype=torch_dtype(otype))), f64(x), vw, k, xtype, otype)


@pytest.mark.parametrize("xtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 64, 7168), (4, 40, 1057), (16, 100, 2048), (33, 70, 1024), (70, 33, 900), (10, 4099, 1057),
                                   (11, 12290, 800)])
def test_integers_are_exact(m, n, k, xtype):
    """Small whole numbers: every partial sum is a multiple of 1/2 below 2^23, so nothing rounds and every product counts."""
    import torch
    rng = np.random.default_rng(k)
    x = rng.integers(-9, 10, (m, k)).astype(np.float64)
    code = rng.integers(0, 16, (n, -(-k // 256) * 256)).astype(np.uint8)
    code[:, k:] = 0
    byte = rng.integers(127, 130, (-(-k // 256), n, 8)).astype(np.uint8)
    q = code[:, 0::2] | (code[:, 1::2] << 4)
    t = torch.from_numpy(x).to(torch_dtype(xtype)).cuda()
    got = fb.gemv_mxfp4(t, torch.from_numpy(q).cuda(), torch.from_numpy(byte).cuda(), dtype=torch.float32)
    assert np.array_equal(f64(got), x @ mxfp4.values(q, byte, k).T)


@pytest.mark.parametrize("xtype", ["float16", "float32"])
def test_activations_are_not_rounded(xtype):
    """Against the unit matrix every element comes back as it is."""
    import torch
    k = 320
    w, ws = mxfp4.quantise(np.eye(k))
    x = matrix(1, 40, k, xtype)
    x[0, :8] = torch.tensor([1.0009765625, -1.9990234375, 6.1035e-05, 5.96e-08, 65504.0, 0.333251953125, -0.0, 2.0 ** -14]).to(x.dtype)
    if xtype == "float32":
        x[1, :6] = torch.tensor([1 + 2.0 ** -23, 3.4028234e38, -3.4028234e38, 16777215.0, 1e-30, 2 - 2.0 ** -23])
    got = fb.gemv_mxfp4(x, torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
    assert torch.equal(got, x)


@pytest.mark.parametrize("xtype", DTYPES)
def test_scales_at_the_ends(xtype):
    """Scale bytes from 0 (2^-127) up to 252 (2^125, the largest with which every code is below 2^128) and every code,
    against one column of x; results below float32's normal range are only held to its smallest normal number."""
    import torch
    k, n = 256, 256
    code = np.tile(np.arange(16, dtype=np.uint8), (n, 16))
    q = code[:, 0::2] | (code[:, 1::2] << 4)
    byte = np.broadcast_to(np.minimum(np.arange(n), 252)[None, :, None], (1, n, 8)).astype(np.uint8)
    vw = mxfp4.values(q, byte, k)
    x = np.zeros((16, k))
    x[np.arange(16), np.arange(16)] = np.where(np.arange(16) % 2, 1536.0, -768.0)
    t = torch.from_numpy(x).to(torch_dtype(xtype)).cuda()
    got = f64(fb.gemv_mxfp4(t, torch.from_numpy(q).cuda(), torch.from_numpy(byte.copy()).cuda(), dtype=torch.float32))
    want = x @ vw.T
    big = np.abs(want) > 3.4028235e38
    assert np.isinf(got[big]).all()
    check("out", got[~big], want[~big], 2.0 ** -126 * (np.abs(want[~big]) < 2.0 ** -126))


def test_nan_scale_and_special_values():
    """A tile marked NaN makes its weight row's results NaN; NaN and infinity of x reach their own row; padding behind k
    takes no part."""
    import torch
    k, n = 300, 40
    w, ws, vw = operand(5, n, k)
    ws = ws.clone()
    ws[1, 7, 0] = 0xFF
    for xtype in DTYPES:
        x = matrix(6, 20, k, xtype)
        x[3, 299], x[5, 0] = float("nan"), float("inf")
        got = f64(fb.gemv_mxfp4(x, w, ws))
        assert np.isnan(got[:, 7]).all() and np.isnan(got[3]).all()
        rest = [i for i in range(20) if i not in (3, 5)]
        assert np.isfinite(np.delete(got[rest], 7, 1)).all()
        vw0 = np.delete(vw, 7, 0)[:, 0]
        row = np.delete(got[5], 7)
        assert np.isnan(row[vw0 == 0]).all() and (row[vw0 != 0] == np.sign(vw0[vw0 != 0]) * np.inf).all()


def test_padded_codes_and_outputs():
    """Codes with rows of their own distance, scales with a larger ld, an output inside a larger one."""
    import torch
    m, n, k = 9, 70, 500
    w, ws, vw = operand(7, n, k)
    wide = torch.full((n, w.shape[1] + 48), 0x77, dtype=torch.uint8, device="cuda")
    wide[:, :w.shape[1]] = w
    more = torch.full((ws.shape[0], n + 5, 8), 0xFF, dtype=torch.uint8, device="cuda")
    more[:, :n] = ws
    x = matrix(8, m, k)
    buf = torch.full((m + 1, n + 11), 7.0, dtype=torch.bfloat16, device="cuda")
    fb.gemv_mxfp4(x, wide[:, :w.shape[1]], more[:, :n], out=buf[:m, 3:3 + n])
    assert torch.equal(buf[:m, 3:3 + n], fb.gemv_mxfp4(x, w, ws))
    assert (buf[:, :3] == 7).all() and (buf[:, 3 + n:] == 7).all() and (buf[m:] == 7).all()


def test_a_row_does_not_depend_on_the_others():
    """The same at every call, and rows of a pass of 16 are those of a call of their own."""
    import torch
    w, ws, _ = operand(9, 200, 1500)
    x = matrix(10, 80, 1500)
    whole = fb.gemv_mxfp4(x, w, ws)
    assert torch.equal(whole, fb.gemv_mxfp4(x, w, ws))
    for lo in (0, 16, 64):
        assert torch.equal(fb.gemv_mxfp4(x[lo:lo + 16], w, ws), whole[lo:lo + 16])
    off = torch.tensor([0, 80], dtype=torch.int32, device="cuda")
    grouped = fb.grouped_gemv_mxfp4(off, x, w[None], ws[None])
    for lo in (0, 16, 64):
        part = torch.tensor([0, 16], dtype=torch.int32, device="cuda")
        assert torch.equal(fb.grouped_gemv_mxfp4(part, x[lo:lo + 16], w[None], ws[None]), grouped[lo:lo + 16])


def experts(seed, groups, n, k):
    import torch
    parts = [operand(seed + e, n, k) for e in range(groups)]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]), [p[2] for p in parts]


@pytest.mark.parametrize("xtype", DTYPES)
@pytest.mark.parametrize("counts,n,k", [([1], 32, 64), ([0, 0, 1], 16, 257), ([3, 0, 17, 1], 100, 600), ([70, 1, 0, 33], 50, 1057),
                                        ([0] * 20 + [2] * 12, 2048, 512), ([0, 0], 16, 32), ([17, 0, 3, 1, 40], 4100, 300),
                                        ([9, 0, 1, 2, 33, 0, 4, 6, 1, 2], 2050, 300)])
def test_experts(counts, n, k, xtype):
    import torch
    log(f"grouped gemv {counts[:6]} {n}x{k} {xtype}")
    groups = len(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows, tokens = int(off[-1]) + 4, 13
    w, ws, vw = experts(11, groups, n, k)
    rng = np.random.default_rng(k)
    src = rng.integers(0, tokens, rows).astype(np.int32)
    src[rng.random(rows) < 0.1] = -1
    src[rng.random(rows) < 0.1] = tokens + 3
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    x = matrix(12, tokens, k, xtype, ld=k + 1)
    picked = np.where(((src >= 0) & (src < tokens))[:, None], f64(x)[np.clip(src, 0, tokens - 1)], 0.0)
    own = torch.from_numpy(picked).to(x.dtype).cuda()
    for use in (True, False):
        out = torch.full((rows, n), 7.0, dtype=x.dtype, device="cuda")
        got = f64(fb.grouped_gemv_mxfp4(dev(off), x if use else own, w, ws, src=dev(src) if use else None, out=out))
        for e in range(groups):
            lo, hi = off[e], off[e + 1]
            if lo < hi:
                check_product(got[lo:hi], picked[lo:hi], vw[e], k, xtype, xtype)
        assert (got[off[-1]:] == 7).all()


@pytest.mark.parametrize("xtype", ["bfloat16", "float16"])
def test_many_experts_of_a_long_k(xtype):
    """Each expert's weight is the first one's with its rows moved on."""
    import torch
    counts, n, k = [1, 0, 3, 18, 2, 5, 1, 0, 33, 4, 8, 9, 1, 1, 16], 4000, 5200
    log(f"grouped gemv {n}x{k} {xtype}")
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    w, ws, vw = operand(40, n, k)
    wide = torch.stack([w.roll(7 * e, 0) for e in range(len(counts))])
    scales = torch.stack([ws.roll(7 * e, 1) for e in range(len(counts))])
    x = matrix(15, int(off[-1]), k, xtype)
    got = f64(fb.grouped_gemv_mxfp4(torch.from_numpy(off).cuda(), x, wide, scales))
    for e in range(len(counts)):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            check_product(got[lo:hi], f64(x)[lo:hi], np.roll(vw, 7 * e, 0), k, xtype, xtype)


def test_offsets_out_of_range_are_clamped():
    import torch
    w, ws, vw = experts(20, 3, 32, 100)
    x = matrix(13, 10, 100)
    out = torch.full((10, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([-5, 4, 2, 1 << 30], dtype=torch.int32, device="cuda")
    got = f64(fb.grouped_gemv_mxfp4(off, x, w, ws, out=out))
    check_product(got[:2], f64(x)[:2], vw[0], 100, "bfloat16", "bfloat16")


def test_weights_past_4_gib():
    """The last expert's codes begin more than 2^32 bytes in."""
    import torch
    groups, n, k = 5, 1 << 18, 7168
    codes, scales, values = operand(30, 64, k)
    w = torch.zeros((groups, n, codes.shape[1]), dtype=torch.uint8, device="cuda")
    ws = torch.zeros((groups, scales.shape[0], n, 8), dtype=torch.uint8, device="cuda")
    w[-1, -64:], ws[-1, :, -64:] = codes, scales
    x = matrix(14, 2, k)
    off = torch.tensor([0, 0, 0, 0, 1, 2], dtype=torch.int32, device="cuda")
    got = fb.grouped_gemv_mxfp4(off, x, w, ws)
    check_product(f64(got[1:, -64:]), f64(x)[1:], values, k, "bfloat16", "bfloat16")
    assert (got[0] == 0).all() and (got[1, :-64] == 0).all()


def test_tiny_fp32_values_end_at_2_to_the_minus_133():
    """Bits of an fp32 x below 2^-133, the smallest of bf16, are cut off; what is above them counts in full."""
    import torch
    k = 512
    rng = np.random.default_rng(31)
    x = np.ldexp(rng.uniform(1, 2, (16, k)) * rng.choice([-1, 1], (16, k)), rng.integers(-149, -100, (16, k))).astype(np.float32)
    x[0, :6] = np.ldexp(np.float32([1, 1, 1.5, 1.9921875, -1, 1.0000001]), [-140, -133, -132, -127, -149, -126])
    w, ws = mxfp4.quantise(np.eye(k) * 2.0 ** 100)
    got = f64(fb.gemv_mxfp4(torch.from_numpy(x).cuda(), torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda()))
    kept = np.trunc(np.ldexp(x.astype(np.float64), 133))
    assert np.array_equal(got, np.ldexp(kept, -33)) and (got[0, :5] == np.ldexp([0, 1, 1.5, 1.984375, 0], [0, -33, -32, -27, 0])).all()


@pytest.mark.parametrize("xtype", DTYPES)
def test_codes_of_2_to_the_128_and_more_are_not_finite(xtype):
    """The weight's values are exact below 2^128: scale bytes up to 252, and the smaller codes of 253 and 254."""
    import torch
    k, n = 256, 64
    q = np.zeros((n, k // 2), np.uint8)
    code = np.tile(np.arange(16, dtype=np.uint8), 4)
    q[:, 0] = code                                                   # element 0; the others are zeros
    byte = np.full((1, n, 8), 127, np.uint8)
    byte[0, :, 0] = np.repeat([251, 252, 253, 254], 16)
    vw = mxfp4.values(q, byte, k)[:, 0]
    x = np.zeros((3, k))
    x[:, 0] = [2.0 ** -10, -3.0 * 2.0 ** -10, 0.0]
    got = f64(fb.gemv_mxfp4(torch.from_numpy(x).to(torch_dtype(xtype)).cuda(), torch.from_numpy(q).cuda(),
                            torch.from_numpy(byte).cuda(), dtype=torch.float32))
    big = np.abs(vw) >= 2.0 ** 128
    assert big.sum() == 4 + 8 and not big[:32].any()
    assert np.array_equal(got[:, ~big], np.outer(x[:, 0], vw[~big]))
    assert not np.isfinite(got[:, big]).any()


@pytest.mark.parametrize("xtype", DTYPES)
def test_each_clamped_expert_has_its_rows(xtype):
    """Offsets below zero and beyond the rows: one writer for every row, nothing behind them touched."""
    import torch
    w, ws, vw = experts(50, 4, 48, 600)
    x = matrix(51, 30, 600, xtype)
    buf = torch.full((36, 48), 7.0, dtype=x.dtype, device="cuda")
    off = torch.tensor([-5, 4, 4, 13, 1 << 30], dtype=torch.int32, device="cuda")
    got = f64(fb.grouped_gemv_mxfp4(off, x, w, ws, out=buf[2:32]))
    for e, (lo, hi) in enumerate([(0, 4), (4, 4), (4, 13), (13, 30)]):
        if lo < hi:
            check_product(got[lo:hi], f64(x)[lo:hi], vw[e], 600, xtype, xtype)
    assert (buf[:2] == 7).all() and (buf[32:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 300, 520), (12, 257, 1057), (20, 96, 64)])
def test_gradient_through_the_column_form(m, n, k, dtype):
    """dx of out = x w^T is the product of dout with the weight quantised along its columns."""
    log(f"gemv gradient {m}x{n}x{k} {dtype}")
    w = matrix(60, n, k, "float32", 0.05)
    _, _, qt, st = fb.quant_mxfp4_1x32(w, rowwise=False, colwise=True)
    values = mxfp4.values(qt.cpu().numpy(), st.cpu().numpy(), n)                # [k, n]
    assert (np.abs(values - f64(w).T) <= np.kron(np.abs(np.pad(f64(w).T, ((0, 0), (0, -n % 32)))).reshape(k, -1, 32).max(2) / 4,
                                                 np.ones((1, 32)))[:, :n]).all()
    dout = matrix(61, m, n, dtype, 0.1)
    check_product(f64(fb.gemv_mxfp4(dout, qt, st)), f64(dout), values, n, dtype, dtype)
    if m > 1:
        import torch
        off = torch.tensor([0, 1, m], dtype=torch.int32, device="cuda")
        got = f64(fb.grouped_gemv_mxfp4(off, dout, torch.stack((qt, qt.flip(0))), torch.stack((st, st.flip(1)))))
        check_product(got[:1], f64(dout)[:1], values, n, dtype, dtype)
        check_product(got[1:], f64(dout)[1:], values[::-1], n, dtype, dtype)
