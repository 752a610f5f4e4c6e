"""Tokens to their experts' rows and back, and the gradient, against float64: every type, odd sizes, strides, plans with
dropped choices, padding and rows of no expert."""

import numpy as np
import pytest

import fp8_fine_grained_fp8bq_amd as fb
from oracle import layer
from tests.gpu_util import log
from tests.layer_util import DTYPES, ROW, U, check, f64, matrix, plan, rounded, torch_dtype

pytestmark = pytest.mark.gpu

# tokens, topk, experts, pad, columns
PLANS = [(1, 1, 1, 1, 1), (1, 8, 16, 1, 7168), (3, 2, 4, 128, 8), (5, 12, 20, 1, 33), (70, 3, 7, 32, 257), (33, 8, 256, 1, 130),
         (200, 4, 16, 256, 512), (64, 1, 3, 1, 2049), (333, 6, 40, 1, 1057)]


def gates(seed, tokens, topk, ld=None):
    import torch
    t = torch.full((tokens, ld or topk), float("nan"), device="cuda")
    t[:, :topk] = torch.from_numpy(np.random.default_rng(seed).normal(0.3, 0.5, (tokens, topk))).float()
    return t[:, :topk]


@pytest.mark.parametrize("tokens,topk,experts,pad,cols", PLANS)
@pytest.mark.parametrize("dtype", DTYPES + ("uint8",))
def test_dispatch(tokens, topk, experts, pad, cols, dtype):
    import torch
    log(f"dispatch {tokens}x{cols} top {topk} of {experts} pad {pad} {dtype}")
    (_, src, pos), (_, nsrc, npos) = plan(tokens, tokens, topk, experts, pad)
    rows = len(nsrc)
    rng = np.random.default_rng(cols)
    for shift in (0, 1):
        if dtype == "uint8":
            x = torch.from_numpy(rng.integers(0, 256, (tokens, cols + 3 * shift), dtype=np.uint8)).cuda()[:, shift:shift + cols]
            bits = lambda t: t.cpu().numpy()  # noqa: E731
        else:
            x = matrix(1, tokens, cols, dtype, ld=cols + 5 * shift, shift=shift)
            bits = lambda t: t.contiguous().view(torch.int32 if dtype == "float32" else torch.int16).cpu().numpy()  # noqa: E731
        buf = torch.full((rows, cols + 2 * shift + 1), 7, dtype=x.dtype, device="cuda")
        out = buf[:, shift:shift + cols]
        got, s = fb.moe_dispatch(x, src, pos, out=out)
        assert s is None and got.data_ptr() == out.data_ptr()
        unused = bits(torch.full((1, 1), 7, dtype=x.dtype, device="cuda"))[0, 0]
        assert np.array_equal(bits(out), layer.dispatch(bits(x), npos, nsrc, rows, unused))
        around = torch.cat((buf[:, :shift], buf[:, shift + cols:]), 1)
        assert (around == 7).all()


@pytest.mark.parametrize("tokens,topk,experts,pad,cols", [(1, 1, 1, 1, 128), (1, 8, 256, 128, 7168), (300, 8, 32, 128, 1152),
                                                          (70, 3, 7, 1, 1280), (520, 2, 9, 16, 128)])
def test_dispatch_of_codes_with_scales(tokens, topk, experts, pad, cols):
    """The bytes and scales are those of the tokens; the scales' ld and the entries around them are left alone."""
    import torch
    log(f"dispatch of codes {tokens}x{cols} top {topk} of {experts} pad {pad}")
    (_, src, pos), (_, nsrc, npos) = plan(7, tokens, topk, experts, pad)
    rows = len(nsrc)
    q, s = fb.quant_act_1x128(matrix(2, tokens, cols))
    wide = torch.full((cols // 128, tokens + 9), float("nan"), device="cuda")
    wide[:, :tokens] = s
    out = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda")
    so = torch.full((cols // 128, rows + 4), 7.0, device="cuda")
    fb.moe_dispatch(q, src, pos, s=wide[:, :tokens], out=out, s_out=so[:, :rows])
    assert np.array_equal(out.cpu().numpy(), layer.dispatch(q.cpu().numpy(), npos, nsrc, rows, 0x55))
    assert np.array_equal(so[:, :rows].t().cpu().numpy(), layer.dispatch(s.t().cpu().numpy(), npos, nsrc, rows, 7.0))
    assert (so[:, rows:] == 7).all()
    a, b = fb.moe_dispatch(q, src, pos, s=s)
    used = nsrc != fb.ROW_UNUSED
    assert np.array_equal(a.cpu().numpy()[used], out.cpu().numpy()[used]) and torch.equal(b[:, used], so[:, :rows][:, used])


@pytest.mark.parametrize("tokens,topk,experts,pad,cols", PLANS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_combine(tokens, topk, experts, pad, cols, dtype):
    import torch
    log(f"combine {tokens}x{cols} top {topk} of {experts} pad {pad} {dtype}")
    (_, src, pos), (_, nsrc, npos) = plan(tokens + 1, tokens, topk, experts, pad, drop=0.3)
    rows = len(nsrc)
    for shift in (0, 1):
        y = matrix(3, rows, cols, dtype, ld=cols + 3 * shift, shift=shift)
        y[torch.from_numpy(nsrc < 0).cuda()] = float("nan")        # rows without a token are not looked at
        base = matrix(4, tokens, cols, dtype, ld=cols + 5 * shift, shift=2 * shift)
        w = gates(5, tokens, topk, topk + shift)
        w[pos < 0] = float("nan")                                  # nor the weight of a choice without a row
        for ww, bb in ((w, None), (w, base), (None, base), (None, None)):
            got = fb.moe_combine(y, pos, ww, base=bb)
            want, mag = layer.combine(f64(y), npos, None if ww is None else f64(ww), None if bb is None else f64(bb))
            check("out", f64(got), want, rounded(want, (topk + 1) * U * mag, dtype))
        again = base.clone().contiguous()
        assert fb.moe_combine(y, pos, w, base=again, out=again).data_ptr() == again.data_ptr()
        assert torch.equal(again, fb.moe_combine(y, pos, w, base=base))       # over the base


@pytest.mark.parametrize("tokens,topk,experts,pad,cols", PLANS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_combine_gradient(tokens, topk, experts, pad, cols, dtype):
    import torch
    log(f"combine gradient {tokens}x{cols} top {topk} of {experts} pad {pad} {dtype}")
    (_, src, pos), (_, nsrc, npos) = plan(tokens + 2, tokens, topk, experts, pad, drop=0.3)
    rows = len(nsrc)
    for shift in (0, 1):
        y = matrix(6, rows, cols, dtype, ld=cols + shift, shift=shift)
        y[torch.from_numpy(nsrc < 0).cuda()] = float("nan")
        dout = matrix(7, tokens, cols, dtype, 0.1, ld=cols + 3 * shift, shift=3 * shift)
        w = gates(8, tokens, topk, topk + shift)
        w[pos < 0] = float("nan")
        buf = torch.full((rows, cols + shift), 7.0, dtype=y.dtype, device="cuda")
        dy, dw = fb.moe_combine_grad(dout, y, pos, w, src, out=buf[:, shift:])
        wy, ww, mag = layer.combine_grad(f64(dout), f64(y), npos, f64(w))
        wy[nsrc == fb.ROW_UNUSED] = 7.0
        check("dy", f64(dy), wy, rounded(wy, U * np.abs(wy), dtype) * (nsrc >= 0)[:, None])
        check("dweight", f64(dw), ww, ROW * mag)
        assert (dw[pos < 0] == 0).all() and (buf[:, :shift] == 7).all()


def test_plans_of_nothing():
    """Every choice another GPU's: no row is written but padding, every token gets its base, or zeros."""
    import torch
    idx = torch.full((6, 3), -1, dtype=torch.int32, device="cuda")
    _, _, src, pos = fb.moe_plan(idx, 4, 32)
    x = matrix(9, 6, 96)
    rows = torch.full((len(src), 96), 7.0, dtype=torch.bfloat16, device="cuda")
    fb.moe_dispatch(x, src, pos, out=rows)
    assert (rows == 7).all()
    y = torch.full((len(src), 96), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert torch.equal(fb.moe_combine(y, pos, base=x), x) and (fb.moe_combine(y, pos) == 0).all()
    w = torch.ones((6, 3), device="cuda")
    dy, dw = fb.moe_combine_grad(x, y, pos, w, src, out=rows)
    assert (dy == 7).all() and (dw == 0).all()


def test_entries_outside_the_rows_are_skipped():
    """A plan's positions and tokens beyond the tensors are not followed."""
    import torch
    pos = torch.tensor([[0, 5], [1 << 30, -7], [2, -(1 << 31)]], dtype=torch.int32, device="cuda")
    src = torch.tensor([0, 77, 2, -1], dtype=torch.int32, device="cuda")       # four rows, three tokens
    x = matrix(10, 3, 40, "float32")
    rows, _ = fb.moe_dispatch(x, src, pos)
    assert torch.equal(rows[0], x[0]) and torch.equal(rows[2], x[2]) and (rows[1] == 0).all() and (rows[3] == 0).all()
    out = fb.moe_combine(rows, pos)
    assert torch.equal(out[0], x[0]) and (out[1] == 0).all() and torch.equal(out[2], x[2])
    dy, dw = fb.moe_combine_grad(x, rows, pos, torch.ones((3, 2), device="cuda"), src)
    assert torch.equal(dy, rows) and (dw[1] == 0).all() and dw[0, 1] == 0 and dw[0, 0] != 0


def test_special_values_pass():
    """NaN and infinities of a token reach its own results only; a weight of 0 against an infinity is NaN, as in the sum."""
    import torch
    (_, src, pos), (_, nsrc, npos) = plan(3, 20, 2, 5, 8, drop=0)
    x = matrix(11, 20, 72)
    x[4, 3], x[9, 70] = float("nan"), float("inf")
    rows, _ = fb.moe_dispatch(x, src, pos)
    w = gates(12, 20, 2)
    w[9] = 0
    out = f64(fb.moe_combine(rows, pos, w))
    bad = np.zeros(out.shape, bool)
    bad[4, 3] = bad[9, 70] = True
    assert np.isnan(out[bad]).all() and np.isfinite(out[~bad]).all()


def test_gradients_against_differences():
    """dispatch, a product with fixed rows, combine: the chain's value is linear in the tokens and in the gates, so
    differences are exact up to float32's roundings."""
    import torch
    tokens, topk, cols = 30, 3, 64
    (_, src, pos), _ = plan(5, tokens, topk, 6, 16)
    x, d, dout = (matrix(s, tokens, cols, "float32") for s in (13, 14, 15))
    fixed = matrix(16, len(src), cols, "float32")
    fixed[src < 0] = 0
    w, e = gates(17, tokens, topk), gates(18, tokens, topk)
    value = lambda x, w: (fb.moe_combine(fb.moe_dispatch(x, src, pos)[0] * fixed, pos, w).double() * dout.double()).sum().item()  # noqa: E731
    rows = fb.moe_dispatch(x, src, pos)[0] * fixed
    rows[src < 0] = 0
    drows, dw = fb.moe_combine_grad(dout, rows, pos, w, src)
    drows[src < 0] = 0
    dx = fb.moe_combine(drows * fixed, pos)
    terms = lambda a, b: (fb.moe_combine(fb.moe_dispatch(a.abs(), src, pos)[0] * fixed.abs(), pos, b.abs()).double()  # noqa: E731
                          * dout.double().abs()).sum().item()
    big = terms(x, w) + terms(d, w) + terms(x, e)
    assert abs(value(x + d, w) - value(x, w) - (dx.double() * d.double()).sum().item()) <= 8 * (topk + ROW / U) * U * big
    assert abs(value(x, w + e) - value(x, w) - (dw.double() * e.double()).sum().item()) <= 8 * (topk + ROW / U) * U * big


@pytest.mark.parametrize("what", ["codes", "combine"])
def test_rows_past_32_bits(what):
    """More than 2^31 bytes of codes, and more than 2^31 elements of rows."""
    import torch
    log(f"rows past 32 bits: {what}")
    tokens, topk, cols = (40000, 8, 7168)
    gen = torch.Generator(device="cuda").manual_seed(1)
    idx = torch.rand((tokens, 16), generator=gen, device="cuda").argsort(1)[:, :topk].to(torch.int32)
    _, _, src, pos = fb.moe_plan(idx, 16)
    if what == "codes":
        q = torch.randint(0, 256, (tokens, cols), generator=gen, device="cuda", dtype=torch.uint8)
        s = torch.rand((cols // 128, tokens), generator=gen, device="cuda")
        a, b = fb.moe_dispatch(q, src, pos, s=s)
        assert a.numel() > 1 << 31
        for lo in range(0, len(src), 40000):
            at = src[lo:lo + 40000].long()
            assert torch.equal(a[lo:lo + 40000], q[at]) and torch.equal(b[:, lo:lo + 40000], s[:, at])
        return
    y = torch.randint(-8, 9, (len(src), cols), generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    assert y.numel() > 1 << 31
    w = torch.randint(1, 5, (tokens, topk), generator=gen, device="cuda").float()
    out = fb.moe_combine(y, pos, w)                      # sums of integers up to 256: exact in bf16
    dout = torch.randint(-2, 3, (tokens, cols), generator=gen, device="cuda").to(torch.bfloat16)
    dy, dw = fb.moe_combine_grad(dout, y, pos, w, src)
    for lo in range(0, tokens, 4000):
        rows = y[pos[lo:lo + 4000].long()].float()
        part = w[lo:lo + 4000, :, None]
        assert torch.equal(out[lo:lo + 4000].float(), (rows * part).sum(1))
        assert torch.equal(dw[lo:lo + 4000], (rows * dout[lo:lo + 4000, None].float()).sum(2))
        assert torch.equal(dy[pos[lo:lo + 4000].long()].float(), part * dout[lo:lo + 4000, None].float())


def test_more_tokens_than_workgroups():
    """More pieces of rows than one launch has workgroups for: dispatch, combine and its gradient of 17 million tokens,
    whose whole numbers come through exactly."""
    import torch
    tokens, cols = 17_000_000, 16
    log(f"rows of {tokens} tokens")
    gen = torch.Generator(device="cuda").manual_seed(2)
    idx = torch.randint(-1, 5, (tokens, 1), generator=gen, device="cuda", dtype=torch.int32)
    _, off, src, pos = fb.moe_plan(idx, 5, 16)
    x = torch.randint(-8, 9, (tokens, cols), generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    rows, _ = fb.moe_dispatch(x, src, pos)
    last = int(off[-1])
    used = src[:last]
    assert torch.equal(rows[:last], torch.where((used >= 0)[:, None], x[used.clamp(min=0).long()], torch.zeros((), dtype=x.dtype, device="cuda")))
    w = torch.randint(1, 4, (tokens, 1), generator=gen, device="cuda").float()
    mine = pos >= 0
    assert torch.equal(fb.moe_combine(rows, pos, w), torch.where(mine, x * w, 0.0).to(x.dtype))
    dy, dw = fb.moe_combine_grad(x, rows, pos, w, src)
    assert torch.equal(dw, torch.where(mine, (x.float() ** 2).sum(1, keepdim=True), 0.0))
    assert torch.equal(fb.moe_combine(dy, pos), torch.where(mine, x * w, 0.0).to(x.dtype))
    assert (dy[:last][used < 0] == 0).all()
