"""RMS norm with the residual's addition and the 1x128 quantisation, and its gradient, against float64: every row shape,
types, strides, special values, and what lies around the outputs."""

import numpy as np
import pytest

import fp8_fine_grained_fp8bq_amd as fb
from oracle import e4m3, layer
from tests.gpu_util import log
from tests.layer_util import DTYPES, ROW, U, check, f64, matrix, rounded, torch_dtype

pytestmark = pytest.mark.gpu

# rstd: half of the sum's error, then the quotient, the sum with eps, the root and the reciprocal
RSTD = ROW / 2 + 4 * U
# y before its rounding: v (one rounding of the sum), rstd, two products
Y = RSTD + 4 * U


def weight(seed, cols, dtype):
    import torch
    return torch.from_numpy(np.random.default_rng(seed + 99).normal(1, 0.4, cols)).to(torch_dtype(dtype)).cuda()


def check_codes(q, s, y, pow2):
    """Codes and scales of the float64 y, each computed value off by at most Y: the scale is that of an amax within Y, the
    code that of a quotient within Y and its own rounding."""
    q, s = q.cpu().numpy(), f64(s).T
    rows, cols = y.shape
    amax = np.abs(y).reshape(rows, cols // 128, 128).max(2)
    if pow2:
        lo, hi = layer.scale(amax * (1 - Y), True), layer.scale(amax * (1 + Y), True)
        assert ((s == lo) | (s == hi)).all()
    else:
        check("scales", s, amax / 448, (Y + U) * amax / 448 + 2.0 ** -150)
    sc = np.repeat(s, 128, 1)
    z = np.abs(np.divide(y, sc, out=np.zeros_like(y), where=sc > 0))
    got = e4m3.decode(q)
    lo, hi = e4m3.decode(e4m3.encode(z * (1 - Y - 2 * U))), e4m3.decode(e4m3.encode(z * (1 + Y + 2 * U)))
    assert ((np.abs(got) >= lo) & (np.abs(got) <= hi)).all()
    assert (np.signbit(got) == np.signbit(y)).all()


def read_back(q, s):
    """Values of E4M3 codes with 1x128 scales."""
    with np.errstate(invalid="ignore"):
        return e4m3.decode(q.cpu().numpy()) * np.repeat(f64(s).T, 128, 1)


def check_forward(x, r, w, eps, out, dtype, pow2=False):
    q, s, y, h, rstd = out
    vx, vr = f64(x), None if r is None else f64(r)
    wh, wr, wy = layer.rmsnorm(vx, vr, f64(w), eps)
    check("rstd", f64(rstd), wr, RSTD * wr)
    if r is not None:
        check("h", f64(h), wh, rounded(wh, U * np.abs(wh), dtype))
    else:
        assert h is None
    if y is not None:
        check("y", f64(y), wy, rounded(wy, Y * np.abs(wy) + 2.0 ** -149, dtype))
    if q is not None:
        check_codes(q, s, wy, pow2)


SHAPES = [(1, 128), (1, 7168), (17, 128), (33, 256), (5, 512), (3, 640), (9, 1024), (6, 4096), (4, 4224), (3, 8192), (3, 8320),
          (2, 16384), (2, 16512), (2, 32768), (4500, 128), (1200, 640)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_into_codes(rows, cols, dtype):
    log(f"norm {rows}x{cols} {dtype}")
    for residual in (False, True):
        x, w = matrix(1, rows, cols, dtype), weight(1, cols, dtype)
        r = matrix(2, rows, cols, dtype, 2.0) if residual else None
        for pow2 in (False, True):
            out = fb.rmsnorm(x, w, 1e-6, residual=r, norm=pow2, pow2=pow2)
            assert (out[2] is None) == (not pow2)
            check_forward(x, r, w, 1e-6, out, dtype, pow2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [1, 2, 7, 8, 9, 33, 127, 129, 135, 511, 513, 520, 1057, 4103, 8199, 16391, 20001])
def test_plain_norm_of_odd_rows(cols, dtype):
    """Any column count, rows that start at any element, each type of weight."""
    rows = 19
    for i, wtype in enumerate(DTYPES):
        log(f"plain norm {rows}x{cols} {dtype} weight {wtype}")
        x = matrix(3, rows, cols, dtype, ld=cols + 3 * i, shift=i)
        r = matrix(4, rows, cols, dtype, ld=cols + 5, shift=2 * i + 1) if i else None
        w = weight(2, cols, wtype)
        out = fb.rmsnorm(x, w, 1e-5, residual=r, quant=False, norm=True)
        assert out[0] is None and out[1] is None
        check_forward(x, r, w, 1e-5, out, dtype)


def test_results_are_the_same_at_every_call_and_row():
    """A row's result does not depend on the rows around it."""
    import torch
    x, w = matrix(5, 300, 1152), weight(3, 1152, "bfloat16")
    a = fb.rmsnorm(x, w, norm=True)
    for lo, hi in ((0, 300), (7, 8), (100, 260)):
        b = fb.rmsnorm(x[lo:hi], w, norm=True)
        assert torch.equal(a[0][lo:hi], b[0]) and torch.equal(a[1][:, lo:hi], b[1])
        assert torch.equal(a[2][lo:hi], b[2]) and torch.equal(a[4][lo:hi], b[4])


def test_codes_of_a_power_of_two_times_the_weight_scale_with_it():
    """Scaling the weight by 2 changes scales only."""
    import torch
    x, w = matrix(6, 40, 512), weight(4, 512, "float32")
    for pow2 in (False, True):
        a, b = fb.rmsnorm(x, w, pow2=pow2), fb.rmsnorm(x, w * 2, pow2=pow2)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1] * 2, b[1])


def test_rows_of_zeros_and_tiny_and_large_values():
    import torch
    rows, cols = 8, 1280
    x = matrix(7, rows, cols, "float32")
    x[0] = 0
    x[1] = -0.0
    x[2] = 1e-30
    x[3] *= 1e16
    x[4, 128:256] = 0                     # one tile of zeros
    x[5] = torch.finfo(torch.float32).tiny
    w = weight(5, cols, "float32")
    w[300] = 0
    for pow2 in (False, True):
        out = fb.rmsnorm(x, w, 1e-6, norm=True, pow2=pow2)
        check_forward(x, None, w, 1e-6, out, "float32", pow2)
        q, s = out[0].cpu().numpy(), f64(out[1])
        zero = 2.0 ** -127 if pow2 else 0.0
        assert (s[:, 0] == zero).all() and (q[0][f64(w) > 0] == 0).all() and (q[0] & 0x7F == 0).all()
        assert (q[1][f64(w) > 0] == 0x80).all()
        assert s[1, 4] == zero and (q[4, 128:256] & 0x7F == 0).all()
    out = fb.rmsnorm(x, w, 0.0, norm=True)
    assert np.isnan(f64(out[2])[0]).all() and np.isnan(read_back(out[0], out[1])[0]).all()         # 0 / 0, as the formula says


@pytest.mark.parametrize("cols", [128, 512, 1152, 16384])
@pytest.mark.parametrize("pow2", [False, True])
def test_nan_and_infinity_stay_in_their_row(cols, pow2):
    x, w = matrix(8, 20, cols), weight(6, cols, "bfloat16")
    clean = fb.rmsnorm(x, w, norm=True, pow2=pow2)
    x = x.clone()
    x[3, 5] = float("nan")
    x[11, cols - 1] = float("inf")
    q, s, y, _, rstd = fb.rmsnorm(x, w, norm=True, pow2=pow2)
    keep = [i for i in range(20) if i not in (3, 11)]
    assert np.array_equal(f64(y)[keep], f64(clean[2])[keep])
    assert np.array_equal(q.cpu().numpy()[keep], clean[0].cpu().numpy()[keep])
    assert np.array_equal(f64(s)[:, keep], f64(clean[1])[:, keep])
    vy, vr, back = f64(y), f64(rstd), read_back(q, s)
    assert np.isnan(vy[3]).all() and np.isnan(vr[3]) and np.isnan(back[3]).all()
    assert vr[11] == 0 and np.isnan(vy[11, -1]) and (vy[11, :-1] == 0).all()
    assert np.isnan(back[11, -1]) and (back[11, :-128] == 0).all()


def test_pointer_level_in_place_and_padded():
    """h over the residual, outputs with rows of their own distance: nothing between the rows is touched, the rows are
    those of the tensor layer."""
    import torch
    rows, cols, ld = 37, 896, 1024
    x, r, w = matrix(9, rows, cols), matrix(10, rows, cols), weight(7, cols, "float16")
    want = fb.rmsnorm(x, w, 1e-6, residual=r, norm=True)
    h = torch.full((rows, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    h[:, :cols] = r
    y = torch.full((rows, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((rows, ld), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((cols // 128, 50), 7.0, device="cuda")
    fb.fp8bq_rmsnorm(x.data_ptr(), fb.BF16, rows, cols, x.stride(0), h.data_ptr(), ld, w.data_ptr(), fb.FP16, 1e-6, h.data_ptr(),
                     ld, y.data_ptr(), ld, q.data_ptr(), ld, s.data_ptr(), 50, None, 0, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(h[:, :cols], want[3]) and torch.equal(y[:, :cols], want[2]) and torch.equal(q[:, :cols], want[0])
    assert torch.equal(s[:, :rows], want[1])
    assert (h[:, cols:] == 7).all() and (y[:, cols:] == 7).all() and (q[:, cols:] == 0x55).all() and (s[:, rows:] == 7).all()


def test_rows_past_32_bits():
    """Rows a million elements apart: offsets beyond 2^31."""
    import torch
    rows, cols, ld = 2300, 256, 1 << 20
    big = torch.zeros((rows, ld), dtype=torch.bfloat16, device="cuda")
    x = matrix(11, rows, cols)
    big[:, :cols] = x
    w = weight(8, cols, "float32")
    a, b = fb.rmsnorm(x, w, residual=x), fb.rmsnorm(big[:, :cols], w, residual=big[:, :cols])
    assert all(torch.equal(p, q) for p, q in zip(a, b) if p is not None)
    a, b = fb.rmsnorm_grad(x, x, w, a[4]), fb.rmsnorm_grad(big[:, :cols], big[:, :cols], w, b[4])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("rows,cols", [(68_000_000, 9), (17_500_000, 130), (4_300_000, 520)])
def test_more_rows_than_workgroups(rows, cols):
    """Rows by 16 lanes, by a wave and by a workgroup, more than one launch has workgroups for: the same as of a slice."""
    import torch
    log(f"norm of {rows} x {cols}")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w = weight(14, cols, "float32")
    _, _, y, _, rstd = fb.rmsnorm(x, w, quant=False, norm=True)
    for lo in (0, rows // 2 - 77, rows - 300):
        a = fb.rmsnorm(x[lo:lo + 300], w, quant=False, norm=True)
        assert torch.equal(y[lo:lo + 300], a[2]) and torch.equal(rstd[lo:lo + 300], a[4])
    dx, dw = fb.rmsnorm_grad(y, x, w, rstd)
    for lo in (0, rows - 300):
        assert torch.equal(dx[lo:lo + 300], fb.rmsnorm_grad(y[lo:lo + 300], x[lo:lo + 300], w, rstd[lo:lo + 300])[0])
    assert torch.isfinite(dw).all()


def check_grad(dy, h, w, rstd, dh, got, dtype):
    vy, vh, vw, vr = f64(dy), f64(h), f64(w), f64(rstd)[:, None]
    wx, ww = layer.rmsnorm_grad(vy, vh, vw, f64(rstd), None if dh is None else f64(dh))
    hat, g = vh * vr, vy * vw
    mean = np.abs(g * hat).mean(1, keepdims=True)
    # the mean is off by ROW and three roundings of each term, the difference and its product by six more
    before = (ROW + 8 * U) * vr * (np.abs(g) + np.abs(hat) * mean) + U * np.abs(wx)
    check("dx", f64(got[0]), wx, rounded(wx, before, dtype))
    # groups of rows added one after the other, then the groups: at most rows + 600 additions, never more than one a row and
    # one a group
    rows = len(vy)
    check("dweight", f64(got[1]), ww, (rows + 600) * U * np.abs(vy * hat).sum(0) + 2.0 ** -149)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7168), (2, 9), (19, 127), (64, 128), (5000, 128), (33, 130), (4100, 300), (50, 512),
                                       (7, 520), (1500, 1057), (333, 2048), (40, 4096), (20, 4104), (600, 7168), (5, 8200),
                                       (9, 16384), (3, 20001), (2, 32768)])
def test_gradient(rows, cols, dtype):
    log(f"norm gradient {rows}x{cols} {dtype}")
    h, dy = matrix(12, rows, cols, dtype), matrix(13, rows, cols, dtype, 0.1)
    w = weight(9, cols, dtype)
    rstd = fb.rmsnorm(h, w, quant=False, norm=True)[4]
    for dh in (None, matrix(14, rows, cols, dtype, 0.1)):
        check_grad(dy, h, w, rstd, dh, fb.rmsnorm_grad(dy, h, w, rstd, dh), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_of_rows_at_any_address(dtype):
    rows, cols = 70, 777
    for i, wtype in enumerate(DTYPES):
        h = matrix(15, rows, cols, dtype, ld=cols + i, shift=i)
        dy, dh = matrix(16, rows, cols, dtype, ld=cols + 7, shift=1), matrix(17, rows, cols, dtype, ld=cols + 2, shift=3)
        w = weight(10, cols, wtype)
        rstd = fb.rmsnorm(h, w, quant=False, norm=True)[4]
        check_grad(dy, h, w, rstd, dh, fb.rmsnorm_grad(dy, h, w, rstd, dh), dtype)


def test_gradient_against_differences():
    """Of the library's own forward pass, in fp32 along random directions. Central differences of step t are off by t^2 / 6
    times the third derivative, which of dy . w h / |h| along d is at most 6 |dy| max|w| |d|^3 / |h|^2 a row (|d| is less
    than |h| here, max|w| less than 2.5), and by the two values' roundings over 2 t."""
    import torch
    rng = np.random.default_rng(3)
    rows, cols, step = 6, 256, 2.0 ** -6
    x, dy, d = (torch.from_numpy(rng.normal(size=(rows, cols))).float().cuda() for _ in range(3))
    r = x.clone()                                             # h = 2 x
    w = weight(11, cols, "float32")
    _, _, y, h, rstd = fb.rmsnorm(x, w, residual=r, norm=True)
    assert (h.norm(dim=1) > d.norm(dim=1)).all() and w.abs().max() < 2.5
    dx, dw = fb.rmsnorm_grad(dy, h, w, rstd)
    value = lambda x, w: (fb.rmsnorm(x, w, residual=r, quant=False, norm=True)[2].double() * dy.double()).sum().item()  # noqa: E731
    noise = Y * (y.double() * dy.double()).abs().sum().item() / step
    size = (dy.double().norm(dim=1) * d.double().norm(dim=1)).sum().item()
    got = (value(x + step * d, w) - value(x - step * d, w)) / (2 * step)
    assert abs(got - (dx.double() * d.double()).sum().item()) <= 2.5 * step ** 2 * size + 1.1 * noise
    e = torch.from_numpy(rng.normal(size=cols)).float().cuda()
    got = (value(x, w + step * e) - value(x, w - step * e)) / (2 * step)       # y is linear in the weight
    assert abs(got - (dw.double() * e.double()).sum().item()) <= 1.1 * noise


def test_gradient_in_place_and_padded():
    import torch
    rows, cols, ld = 45, 600, 640
    h, dy, dh, w = matrix(18, rows, cols), matrix(19, rows, cols), matrix(20, rows, cols), weight(12, cols, "bfloat16")
    rstd = fb.rmsnorm(h, w, quant=False, norm=True)[4]
    want = fb.rmsnorm_grad(dy, h, w, rstd, dh)
    ws = torch.empty(fb.fp8bq_rmsnorm_grad_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    for over in ("dh", "dy"):
        buf = torch.full((rows, ld), 7.0, dtype=torch.bfloat16, device="cuda")
        buf[:, :cols] = dh if over == "dh" else dy
        dw = torch.full((cols + 8,), 7.0, device="cuda")
        p = lambda name, t: (buf.data_ptr(), ld) if over == name else (t.data_ptr(), t.stride(0))  # noqa: E731
        (a, lda), (b, ldb) = p("dy", dy), p("dh", dh)
        fb.fp8bq_rmsnorm_grad(a, fb.BF16, rows, cols, lda, h.data_ptr(), h.stride(0), w.data_ptr(), fb.BF16, rstd.data_ptr(), b, ldb,
                              buf.data_ptr(), ld, dw.data_ptr(), ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert torch.equal(buf[:, :cols], want[0]) and torch.equal(dw[:cols], want[1])
        assert (buf[:, cols:] == 7).all() and (dw[cols:] == 7).all()


def test_gradient_is_the_same_at_every_call():
    import torch
    h, dy, w = matrix(21, 3000, 768), matrix(22, 3000, 768), weight(13, 768, "float32")
    rstd = fb.rmsnorm(h, w)[4]
    a = fb.rmsnorm_grad(dy, h, w, rstd)
    for _ in range(3):
        b = fb.rmsnorm_grad(dy, h, w, rstd)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def check_read_back(out, wy):
    """Values within half a step of E4M3 of the float64 y, and half of its smallest step (2^-10 s), 1% being for the other
    roundings; 2^-149 for y's own where it is subnormal, and what 448 s leaves of it where the scale is rounded off."""
    back = read_back(out[0], out[1])
    assert np.isfinite(back).all()
    s = np.repeat(f64(out[1]).T, 128, 1)
    check("values", back, wy, 1.01 * (2.0 ** -4 * np.abs(wy) + 2.0 ** -10 * s) + 2.0 ** -149 + np.maximum(np.abs(wy) - 448 * s, 0))


@pytest.mark.parametrize("cols", [128, 512, 1152, 16512])
@pytest.mark.parametrize("residual", [False, True])
def test_weights_whose_product_with_a_row_overflows(cols, residual):
    """h * weight beyond float32's range where y = h * rstd * weight is not."""
    import torch
    x = torch.full((3, cols), 100.0, device="cuda")
    x[1, ::2], x[2, 5] = -37.5, 1e4
    w = torch.ones(cols, device="cuda")
    w[: cols // 2] = 1e37
    w[5], w[7] = 1.0, 1e30
    r = x * 3 if residual else None
    for pow2 in (False, True):
        out = fb.rmsnorm(x, w, 1e-6, residual=r, norm=True, pow2=pow2)
        wy = layer.rmsnorm(f64(x), None if r is None else f64(r), f64(w), 1e-6)[2]
        check("y", f64(out[2]), wy, rounded(wy, Y * np.abs(wy), "float32"))
        check_codes(out[0], out[1], wy, pow2)
        check_read_back(out, wy)


@pytest.mark.parametrize("size", [1e-40, 1e-41, 3e-42, 1e-42, 3e-43, 1e-43])
def test_scales_of_a_few_steps_of_the_smallest_number(size):
    """amax / 448 rounds to a scale up to a third too small: codes end at 448 then."""
    x, w = matrix(24, 40, 640, "float32"), weight(16, 640, "float32") * size
    out = fb.rmsnorm(x, w, 0.0, norm=True)
    wy = layer.rmsnorm(f64(x), None, f64(w), 0.0)[2]
    check("scales", f64(out[1]).T, np.abs(wy).reshape(40, 5, 128).max(2) / 448, 2.0 ** -149)
    check_read_back(out, wy)


@pytest.mark.parametrize("size", [1e-35, 1e-38, 1e-41])
def test_large_rows_with_tiny_weights(size):
    """h * weight is normal, the scale of y is not."""
    x, w = matrix(23, 20, 640, "float32") * 1e15, weight(15, 640, "float32") * size
    out = fb.rmsnorm(x, w, 0.0, norm=True)
    check_read_back(out, layer.rmsnorm(f64(x), None, f64(w), 0.0)[2])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("cols", [128, 512, 1152, 7168])
def test_codes_bit_for_bit(cols, residual, dtype):
    """Given rstd, every step up to the codes and scales is one float32 operation, which numpy does alike."""
    rows = 40
    x, w = matrix(25, rows, cols, dtype), weight(17, cols, dtype)
    x[5, :128] *= 2.0 ** -12                                           # tiles whose scale of h * weight is below 2^-100, from y
    w[:128] *= 1e-28 if dtype == "float32" else 1
    r = matrix(26, rows, cols, dtype, 2.0) if residual else None
    f32 = lambda t: f64(t).astype(np.float32)  # noqa: E731
    tiles = lambda a: a.reshape(rows, -1, 128)  # noqa: E731
    v = f32(x) + f32(r) if residual else f32(x)
    for pow2 in (False, True):
        q, s, _, _, rstd = fb.rmsnorm(x, w, residual=r, pow2=pow2)
        hw, y = tiles(v * f32(w)), tiles(v * f32(rstd)[:, None] * f32(w))
        amax = lambda a: np.abs(a).max(2, keepdims=True)  # noqa: E731
        if pow2:
            want_s = layer.scale(amax(y).astype(np.float64), True).astype(np.float32)
            z = y / want_s
        else:
            of_hw, of_y = amax(hw) / np.float32(448), amax(y) / np.float32(448)
            from_hw = of_hw >= np.float32(2.0 ** -100)
            want_s = np.where(from_hw, of_hw * f32(rstd)[:, None, None], of_y)
            z = np.where(from_hw, hw / of_hw, y / of_y)
        assert z.dtype == np.float32 and want_s.dtype == np.float32
        assert np.array_equal(f32(s).T, want_s[:, :, 0])
        assert np.array_equal(q.cpu().numpy(), e4m3.encode(z.astype(np.float64)).reshape(rows, cols))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [5, 100, 333, 1057, 7168])
def test_sum_over_x_itself(cols, dtype):
    """h over x: what lanes without a column of their own load may be stored over by then."""
    import torch
    rows = 50
    x, r, w = matrix(27, rows, cols, dtype), matrix(28, rows, cols, dtype), weight(18, cols, dtype)
    want = fb.rmsnorm(x, w, 1e-6, residual=r, quant=False, norm=True)
    h, y, rstd = x.clone(), torch.empty_like(want[2]), torch.empty(rows, device="cuda")
    code = DTYPES.index(dtype)
    fb.fp8bq_rmsnorm(h.data_ptr(), code, rows, cols, cols, r.data_ptr(), cols, w.data_ptr(), code, 1e-6, h.data_ptr(), cols,
                     y.data_ptr(), cols, None, 0, None, 0, rstd.data_ptr(), 0, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(h, want[3]) and torch.equal(y, want[2]) and torch.equal(rstd, want[4])


def test_ends_of_the_sum_of_squares():
    """Mean squares beyond float32 give zeros; squares that vanish an infinite rstd without eps, and nothing of note with it."""
    import torch
    x = torch.full((3, 256), 1e20, device="cuda")
    x[1], x[2] = 1e-25, 1e-18
    w = weight(19, 256, "float32")
    q, s, y, _, rstd = fb.rmsnorm(x, w, 0.0, norm=True)
    assert rstd[0] == 0 and (y[0] == 0).all() and (read_back(q, s)[0] == 0).all()
    assert torch.isinf(rstd[1]) and torch.isinf(y[1]).all()
    check("rstd", f64(rstd[2:]), np.array([1e18]), 1e18 * (RSTD + 256 * 2.0 ** -150 / 256e-36))
    check_forward(x[1:], None, w, 1e-12, fb.rmsnorm(x[1:], w, 1e-12, norm=True), "float32")
