"""The C entry points and the tensor layer of the operators around a layer's Linears: bad arguments are refused with the
documented status before any GPU call, with a message. Runs without a GPU."""

import ctypes
import os

import pytest

import fp8_fine_grained_fp8bq_amd as fb

A16, S8, O4 = 0x10000, 0x20008, 0x30004       # aligned to 16, 8, 4 (never dereferenced)
BIG = (1 << 63) - 1
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fb.LIB_PATH):
        pytest.skip("libfp8bq.so not built (run __graft_entry__.build())")
    return fb.lib()


def expect(L, status, fn, args, **change):
    """Calls fn with the good arguments changed at the given positions (a3=... is argument 3)."""
    args = list(args)
    for k, v in change.items():
        args[int(k[1:])] = v
    assert getattr(L, fn)(*args) == status, (fn, change, L.fp8bq_last_error())
    assert L.fp8bq_last_error()


#       x    t  rows cols ld   r    ldr  w   wt eps   h    ldh  y    ldy  q    ldq  s   lds rstd fl
NORM = [A16, 0, 70, 256, 256, A16, 256, A16, 2, 1e-6, A16, 256, A16, 256, A16, 256, O4, 70, O4, 0, None]
NORMG = [A16, 0, 70, 256, 256, A16, 256, A16, 2, O4, A16, 256, A16, 256, O4, O4, None]
DISP = [A16, 1, 50, 256, 256, O4, 50, O4, 4, O4, 300, A16, 256, O4, 300, None]
COMB = [A16, 0, 300, 256, 256, O4, 50, 4, O4, 4, A16, 256, A16, 256, None]
COMBG = [A16, 0, 50, 256, 256, A16, 300, 256, O4, 4, O4, 4, O4, A16, 256, O4, None]
GEMV = [7, 90, 300, A16, 0, 300, A16, 256, S8, 90, A16, 0, 90, None]
GROUPED = [4, O4, 70, 90, 300, A16, 0, 20, 300, O4, A16, 256, S8, 90, A16, 0, 90, None]
ALL = {"fp8bq_rmsnorm": NORM, "fp8bq_rmsnorm_grad": NORMG, "fp8bq_moe_dispatch": DISP, "fp8bq_moe_combine": COMB,
       "fp8bq_moe_combine_grad": COMBG, "fp8bq_gemv_mxfp4": GEMV, "fp8bq_grouped_gemv_mxfp4": GROUPED}


def each(L, status, fn, values, positions):
    for i in positions:
        for v in values:
            expect(L, status, fn, ALL[fn], **{f"a{i}": v})


def test_norm_refusals(L):
    fn = "fp8bq_rmsnorm"
    each(L, fb.E_INVAL, fn, [None], (0, 5, 7, 10, 14, 16))
    expect(L, fb.E_INVAL, fn, NORM, a12=None, a14=None, a16=None)
    each(L, fb.E_INVAL, fn, [0, -1], (2, 3))
    each(L, fb.E_INVAL, fn, [3, -1], (1, 8))
    each(L, fb.E_INVAL, fn, [255, -256], (4, 6, 11, 13, 15))
    each(L, fb.E_INVAL, fn, [-1e-6, NAN, float("inf")], (9,))
    each(L, fb.E_INVAL, fn, [69], (17,))
    each(L, fb.E_INVAL, fn, [1, 0x20], (19,))
    expect(L, fb.E_SHAPE, fn, NORM, a3=250)
    expect(L, fb.E_SHAPE, fn, NORM, a3=32896, a4=40000, a6=40000, a11=40000, a13=40000, a15=40000)
    expect(L, fb.E_SHAPE, fn, NORM, a2=1 << 31, a17=1 << 31)
    each(L, fb.E_SHAPE, fn, [BIG], (4, 6, 11, 13, 15, 17))
    each(L, fb.E_ALIGN, fn, [A16 + 1], (0, 5, 10, 12))
    each(L, fb.E_ALIGN, fn, [A16 + 2], (7, 14, 16, 18))
    expect(L, fb.E_ALIGN, fn, NORM, a14=A16 + 8)
    expect(L, fb.E_ALIGN, fn, NORM, a15=264)


def test_norm_gradient_refusals(L):
    fn = "fp8bq_rmsnorm_grad"
    each(L, fb.E_INVAL, fn, [None], (0, 5, 7, 9, 12, 14, 15))
    each(L, fb.E_INVAL, fn, [0, -1], (2, 3))
    each(L, fb.E_INVAL, fn, [3, -1], (1, 8))
    each(L, fb.E_INVAL, fn, [255], (4, 6, 11, 13))
    expect(L, fb.E_SHAPE, fn, NORMG, a3=32769, a4=40000, a6=40000, a11=40000, a13=40000)
    each(L, fb.E_SHAPE, fn, [BIG], (4, 6, 11, 13))
    each(L, fb.E_ALIGN, fn, [A16 + 1], (0, 5, 7, 10, 12))
    each(L, fb.E_ALIGN, fn, [O4 + 2], (9, 14, 15))
    n = ctypes.c_int64(-1)
    assert L.fp8bq_rmsnorm_grad_workspace_size(4096, 7168, ctypes.byref(n)) == fb.OK and n.value >= 4 * 7168
    assert fb.fp8bq_rmsnorm_grad_workspace_size(1, 1) >= 4
    assert L.fp8bq_rmsnorm_grad_workspace_size(1, 1, None) == fb.E_INVAL
    assert L.fp8bq_rmsnorm_grad_workspace_size(0, 1, ctypes.byref(n)) == fb.E_INVAL
    assert L.fp8bq_rmsnorm_grad_workspace_size(1, 32769, ctypes.byref(n)) == fb.E_SHAPE


def test_dispatch_refusals(L):
    fn = "fp8bq_moe_dispatch"
    each(L, fb.E_INVAL, fn, [None], (0, 5, 7, 9, 11, 13))
    each(L, fb.E_INVAL, fn, [0, 3, 8, 2], (1,))                # 2: scales with 16-bit rows
    each(L, fb.E_INVAL, fn, [0, -1], (2, 3, 8, 10))
    each(L, fb.E_INVAL, fn, [255], (4, 12))
    each(L, fb.E_INVAL, fn, [49], (6,))
    each(L, fb.E_INVAL, fn, [299], (14,))
    expect(L, fb.E_SHAPE, fn, DISP, a3=250)
    each(L, fb.E_SHAPE, fn, [BIG], (2, 3, 4, 6, 8, 10, 12, 14))
    expect(L, fb.E_SHAPE, fn, DISP, a2=1 << 28, a6=1 << 28)
    each(L, fb.E_ALIGN, fn, [O4 + 2], (5, 7, 9, 13))
    plain = DISP[:5] + [None, 0] + DISP[7:13] + [None, 0, None]
    for elem in (2, 4):
        for i in (0, 11):
            expect(L, fb.E_ALIGN, fn, plain, a1=elem, **{f"a{i}": A16 + 1})


def test_combine_refusals(L):
    fn = "fp8bq_moe_combine"
    each(L, fb.E_INVAL, fn, [None], (0, 5, 12))
    each(L, fb.E_INVAL, fn, [3], (1,))
    each(L, fb.E_INVAL, fn, [0, -1], (2, 3, 6, 7))
    each(L, fb.E_INVAL, fn, [255], (4, 11, 13))
    each(L, fb.E_INVAL, fn, [3], (9,))
    each(L, fb.E_SHAPE, fn, [BIG], (2, 3, 4, 6, 7, 9, 11, 13))
    each(L, fb.E_ALIGN, fn, [A16 + 1], (0, 5, 8, 10, 12))


def test_combine_gradient_refusals(L):
    fn = "fp8bq_moe_combine_grad"
    each(L, fb.E_INVAL, fn, [None], (0, 5, 8, 10, 12, 13, 15))
    each(L, fb.E_INVAL, fn, [3], (1,))
    each(L, fb.E_INVAL, fn, [0, -1], (2, 3, 6, 9))
    each(L, fb.E_INVAL, fn, [255], (4, 7, 14))
    each(L, fb.E_INVAL, fn, [3], (11,))
    each(L, fb.E_SHAPE, fn, [BIG], (2, 3, 4, 6, 7, 9, 11, 14))
    each(L, fb.E_ALIGN, fn, [A16 + 1], (0, 5, 8, 10, 12, 13, 15))


@pytest.mark.parametrize("fn", ["fp8bq_gemv_mxfp4", "fp8bq_grouped_gemv_mxfp4"])
def test_product_refusals(L, fn):
    d = 4 if "grouped" in fn else 0                            # positions from b on; x, its type and ld come 2 and 3 later
    m, n, k, x, t, ldx = (2, 3, 4, 5, 6, 8) if d else (0, 1, 2, 3, 4, 5)
    b, ldb, sb, ldsb, out, ot, ldo = (i + d for i in (6, 7, 8, 9, 10, 11, 12))
    each(L, fb.E_INVAL, fn, [None], (x, b, sb, out))
    each(L, fb.E_INVAL, fn, [0, -1], (m, n, k))
    each(L, fb.E_INVAL, fn, [3, -1], (t, ot))
    each(L, fb.E_INVAL, fn, [299], (ldx,))
    each(L, fb.E_INVAL, fn, [89], (ldsb, ldo))
    each(L, fb.E_INVAL, fn, [240], (ldb,))
    each(L, fb.E_SHAPE, fn, [BIG], (m, n, k, ldx, ldo))
    each(L, fb.E_SHAPE, fn, [1 << 40], (ldb, ldsb))
    each(L, fb.E_ALIGN, fn, [A16 + 1], (x, out))
    each(L, fb.E_ALIGN, fn, [A16 + 4], (b, sb))
    each(L, fb.E_ALIGN, fn, [264], (ldb,))
    if d:
        expect(L, fb.E_INVAL, fn, GROUPED, a1=None)
        expect(L, fb.E_INVAL, fn, GROUPED, a7=0)
        expect(L, fb.E_INVAL, fn, GROUPED, a9=None)            # 20 rows of x for 70
        each(L, fb.E_SHAPE, fn, [0, 257, -1], (0,))
        each(L, fb.E_ALIGN, fn, [O4 + 2], (1, 9))
        expect(L, fb.E_SHAPE, fn, GROUPED, a7=1 << 31)


def test_good_arguments_reach_the_device_check(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible; valid arguments would launch")
    for fn, ok in ALL.items():
        expect(L, fb.E_DEVICE, fn, ok)
    expect(L, fb.E_DEVICE, "fp8bq_rmsnorm", NORM, a5=None, a10=None, a12=None, a18=None)
    expect(L, fb.E_DEVICE, "fp8bq_rmsnorm", NORM, a3=33, a14=None, a16=None)
    expect(L, fb.E_DEVICE, "fp8bq_moe_dispatch", DISP, a1=4, a3=33, a5=None, a13=None)
    expect(L, fb.E_DEVICE, "fp8bq_moe_combine", COMB, a8=None, a9=0, a10=None, a11=0)
    expect(L, fb.E_DEVICE, "fp8bq_grouped_gemv_mxfp4", GROUPED, a9=None, a7=70)


def test_tensor_layer_refusals():
    """What the C entry cannot see (types, shapes, strides, places) raises ValueError."""
    import torch
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    w, rstd = torch.ones(256), torch.ones(4)
    src, pos = torch.zeros(9, dtype=torch.int32), torch.zeros((4, 2), dtype=torch.int32)
    gate, y = torch.zeros((4, 2)), torch.zeros((9, 256), dtype=torch.bfloat16)
    codes, scales = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((2, 4))
    q, s = torch.zeros((8, 128), dtype=torch.uint8), torch.zeros((1, 8, 8), dtype=torch.uint8)
    off = torch.zeros(3, dtype=torch.int32)
    gq, gs = q.expand(2, 8, 128).contiguous(), s.expand(2, 1, 8, 8).contiguous()
    good = [lambda: fb.rmsnorm(x, w), lambda: fb.rmsnorm_grad(x, x, w, rstd), lambda: fb.moe_dispatch(x, src, pos),
            lambda: fb.moe_dispatch(codes, src, pos, s=scales), lambda: fb.moe_combine(y, pos, gate, base=x),
            lambda: fb.moe_combine_grad(x, y, pos, gate, src), lambda: fb.gemv_mxfp4(x, q, s),
            lambda: fb.grouped_gemv_mxfp4(off, x, gq, gs, src=src)]
    for f in good:
        with pytest.raises(ValueError, match="on the GPU"):
            f()
    bad = [
        lambda: fb.rmsnorm(x.double(), w),
        lambda: fb.rmsnorm(x.t(), w),
        lambda: fb.rmsnorm(x[0], w),
        lambda: fb.rmsnorm(x[:0], w),
        lambda: fb.rmsnorm(x, w[:255]),
        lambda: fb.rmsnorm(x, torch.ones(512)[::2]),
        lambda: fb.rmsnorm(x, w.double()),
        lambda: fb.rmsnorm(x, w, "small"),
        lambda: fb.rmsnorm(x, w, residual=x.float()),
        lambda: fb.rmsnorm(x, w, residual=x[:3]),
        lambda: fb.rmsnorm(x, w, quant=False),
        lambda: fb.rmsnorm(x[:, :200], w[:200]),
        lambda: fb.rmsnorm_grad(x.float(), x, w, rstd),
        lambda: fb.rmsnorm_grad(x, x[:3], w, rstd),
        lambda: fb.rmsnorm_grad(x, x, w, rstd[:3]),
        lambda: fb.rmsnorm_grad(x, x, w, rstd.double()),
        lambda: fb.rmsnorm_grad(x, x, w, rstd, dh=x.t()),
        lambda: fb.moe_dispatch(x, src.long(), pos),
        lambda: fb.moe_dispatch(x, src, pos[:3]),
        lambda: fb.moe_dispatch(x, src, torch.zeros((4, 4), dtype=torch.int32)[:, ::2]),
        lambda: fb.moe_dispatch(x, src, pos, s=scales),
        lambda: fb.moe_dispatch(x, src, pos, s_out=torch.zeros((2, 9))),
        lambda: fb.moe_dispatch(codes, src, pos, s=scales[:1]),
        lambda: fb.moe_dispatch(codes[:, :200], src, pos, s=scales),
        lambda: fb.moe_dispatch(codes, src, pos, s=scales, s_out=scales),
        lambda: fb.moe_dispatch(x, src, pos, out=y[:8]),
        lambda: fb.moe_dispatch(x, src, pos, out=y.float()),
        lambda: fb.moe_dispatch(x.to(torch.int16), src, pos),
        lambda: fb.moe_combine(y, pos, gate.double()),
        lambda: fb.moe_combine(y, pos, gate[:, :1]),
        lambda: fb.moe_combine(y, pos, gate, base=x.float()),
        lambda: fb.moe_combine(codes, pos),
        lambda: fb.moe_combine(y, pos.long()),
        lambda: fb.moe_combine(y, pos, out=x[:3]),
        lambda: fb.moe_combine_grad(x, y, pos, None, src),
        lambda: fb.moe_combine_grad(x, y, pos, gate, src[:8]),
        lambda: fb.moe_combine_grad(x[:3], y, pos, gate, src),
        lambda: fb.moe_combine_grad(x.float(), y, pos, gate, src),
        lambda: fb.gemv_mxfp4(x, q[:, :64], s),
        lambda: fb.gemv_mxfp4(torch.zeros((4, 257)), q, s),
        lambda: fb.gemv_mxfp4(x, torch.zeros((8, 256), dtype=torch.uint8), torch.zeros((2, 8, 8), dtype=torch.uint8)),
        lambda: fb.gemv_mxfp4(x.int(), q, s),
        lambda: fb.gemv_mxfp4(x, q, s, dtype=torch.int8),
        lambda: fb.gemv_mxfp4(x, q, s, dtype="bf16"),
        lambda: fb.grouped_gemv_mxfp4(off[:2], x, gq, gs),
        lambda: fb.grouped_gemv_mxfp4(off.long(), x, gq, gs),
        lambda: fb.grouped_gemv_mxfp4(off, x, q, s),
        lambda: fb.grouped_gemv_mxfp4(off, x, gq, gs, src=src.long()),
        lambda: fb.grouped_gemv_mxfp4(off, x, gq.transpose(0, 1), gs),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError) as e:
            f()
            print("accepted:", i)
        assert "on the GPU" not in str(e.value), i


def test_message_of_a_refusal():
    with pytest.raises(fb.Fp8bqError, match="E_INVAL.*no output"):
        fb.fp8bq_rmsnorm(A16, 0, 4, 64, 64, None, 0, A16, 0, 1e-6, None, 0, None, 0, None, 0, None, 0, None)


def test_no_rows_reach_the_device_check(L):
    """No expert here got a token: rows 0 with null pointers to the rows, which torch gives empty tensors."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible; valid arguments would launch")
    expect(L, fb.E_DEVICE, "fp8bq_moe_combine", COMB, a0=None, a2=0)
    expect(L, fb.E_DEVICE, "fp8bq_moe_combine", COMB, a0=None, a2=0, a4=0, a8=None, a9=0, a10=None, a11=0)
    expect(L, fb.E_DEVICE, "fp8bq_moe_combine_grad", COMBG, a5=None, a6=0, a12=None, a13=None)
    expect(L, fb.E_DEVICE, "fp8bq_moe_combine_grad", COMBG, a5=None, a6=0, a7=0, a12=None, a13=None, a14=0)
    expect(L, fb.E_INVAL, "fp8bq_moe_combine", COMB, a0=None, a2=-1)
    expect(L, fb.E_INVAL, "fp8bq_moe_combine", COMB, a0=None, a2=0, a3=0)
    expect(L, fb.E_INVAL, "fp8bq_moe_combine", COMB, a0=None, a2=0, a12=None)
    each(L, fb.E_INVAL, "fp8bq_moe_combine_grad", [None], (0, 8, 10, 15))
    off = (ctypes.c_int64 * 3)(0, 0, 0)
    product = [2, off, 256, 384, None, 384, None, 1, A16, 384, O4, 3, None, 256]
    for fn, rest in (("fp8bq_grouped_gemm", [0, None]), ("fp8bq_grouped_gemm_decode", [0, None]),
                     ("fp8bq_grouped_gemm_decode_ws", [None, 0, 0, None]), ("fp8bq_grouped_gemm_decode_noalloc", [0, None])):
        expect(L, fb.E_DEVICE, fn, product + rest)
        each_of = lambda values, i: [expect(L, fb.E_INVAL, fn, product + rest, **{f"a{i}": v}) for v in values]  # noqa: E731
        each_of([None], 8), each_of([None], 10), each_of([383], 5), each_of([383], 9), each_of([255], 13)
        expect(L, fb.E_INVAL, fn, product + rest, a1=(ctypes.c_int64 * 3)(0, 0, 128))


def test_no_rows_in_the_tensor_layer():
    """Empty matrices of rows are no refusal of their own."""
    import torch
    x, pos, gate = torch.zeros((4, 256)), torch.full((4, 2), -1, dtype=torch.int32), torch.zeros((4, 2))
    y, src = torch.zeros((0, 256)), torch.zeros(0, dtype=torch.int32)
    for f in (lambda: fb.moe_combine(y, pos, gate, base=x), lambda: fb.moe_combine_grad(x, y, pos, gate, src)):
        with pytest.raises(ValueError, match="on the GPU"):
            f()
    for f in (lambda: fb.moe_combine(y[:, :0], pos, gate), lambda: fb.moe_combine_grad(x, y, pos, gate, torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError, match="shape|columns|must be"):
            f()
