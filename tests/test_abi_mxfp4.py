"""The C entry points and the tensor layer of the MXFP4 operators and the routing: bad arguments are refused with the
documented status before any GPU call, with a message. Runs without a GPU."""

import ctypes
import os

import pytest

import fp8_fine_grained_fp8bq_amd as fb

A16, S8, O4 = 0x10000, 0x20008, 0x30004       # aligned to 16, 8, 4 (never dereferenced)
BIG = (1 << 63) - 1


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


QUANT = [A16, 0, 70, 300, 300, A16, 256, S8, 70, A16, 128, S8, 300, 0, None]
DISPATCH = [A16, 0, 40, 300, 300, O4, 70, A16, 256, S8, 70, A16, 128, S8, 300, 0, None, None]
DEQUANT = [A16, 70, 300, 256, S8, 70, A16, 0, 300, None]
GEMM = [70, 90, 300, A16, 256, S8, 70, A16, 256, S8, 90, A16, 0, 90, None]
GROUPED = [4, O4] + GEMM
PLAN = [O4, 100, 8, 8, 16, 32, O4, O4, O4, 800 + 16 * 31, O4, O4, None]
BALANCE = [A16, 2, 100, 64, 64, O4, 6, 6, O4, 3, 0, 0.1, O4, O4, O4, O4, None]
GRAD = [O4] + BALANCE[:12] + [O4, O4, A16, 64, None]


@pytest.mark.parametrize("fn,ok", [("fp8bq_quant_mxfp4_1x32", QUANT), ("fp8bq_dispatch_mxfp4_1x32", DISPATCH)])
def test_quant_refusals(L, fn, ok):
    d = 2 if "dispatch" in fn else 0            # positions from the outputs on
    p = lambda i: f"a{i + d}"                   # noqa: E731
    for i in (0, 5 + d, 7 + d, 9 + d, 11 + d):
        expect(L, fb.E_INVAL, fn, ok, **{f"a{i}": None})
    expect(L, fb.E_INVAL, fn, ok, a1=3)
    expect(L, fb.E_INVAL, fn, ok, **{f"a{6 if d else 2}": 0})
    expect(L, fb.E_INVAL, fn, ok, a3=-1)
    expect(L, fb.E_INVAL, fn, ok, a4=299)
    expect(L, fb.E_INVAL, fn, ok, **{p(6): 240})
    expect(L, fb.E_INVAL, fn, ok, **{p(8): 69})
    expect(L, fb.E_INVAL, fn, ok, **{p(10): 112})
    expect(L, fb.E_INVAL, fn, ok, **{p(12): 299})
    expect(L, fb.E_INVAL, fn, ok, **{p(13): 1})
    expect(L, fb.E_INVAL, fn, ok, **{p(5): None, p(7): None, p(9): None, p(11): None})
    expect(L, fb.E_ALIGN, fn, ok, a0=A16 + 1)
    expect(L, fb.E_ALIGN, fn, ok, **{p(5): A16 + 8})
    expect(L, fb.E_ALIGN, fn, ok, **{p(6): 264})
    expect(L, fb.E_ALIGN, fn, ok, **{p(7): S8 + 4})
    expect(L, fb.E_ALIGN, fn, ok, **{p(11): S8 + 4})
    expect(L, fb.E_SHAPE, fn, ok, **{f"a{6 if d else 2}": 1 << 40, p(8): 1 << 41, p(10): 1 << 41})
    expect(L, fb.E_SHAPE, fn, ok, a4=BIG)
    expect(L, fb.E_SHAPE, fn, ok, a3=BIG // 2, a4=BIG)
    if d:
        expect(L, fb.E_INVAL, fn, ok, a5=None)
        expect(L, fb.E_INVAL, fn, ok, a2=0)
        expect(L, fb.E_ALIGN, fn, ok, a5=O4 + 2)
        expect(L, fb.E_ALIGN, fn, ok, a16=A16 + 8)


def test_dequant_refusals(L):
    fn = "fp8bq_dequant_mxfp4_1x32"
    for i in (0, 4, 6):
        expect(L, fb.E_INVAL, fn, DEQUANT, **{f"a{i}": None})
    expect(L, fb.E_INVAL, fn, DEQUANT, a1=0)
    expect(L, fb.E_INVAL, fn, DEQUANT, a3=128)
    expect(L, fb.E_INVAL, fn, DEQUANT, a5=69)
    expect(L, fb.E_INVAL, fn, DEQUANT, a7=7)
    expect(L, fb.E_INVAL, fn, DEQUANT, a8=299)
    expect(L, fb.E_ALIGN, fn, DEQUANT, a0=A16 + 4)
    expect(L, fb.E_ALIGN, fn, DEQUANT, a6=A16 + 1)
    expect(L, fb.E_SHAPE, fn, DEQUANT, a1=BIG, a5=BIG)


@pytest.mark.parametrize("fn,ok", [("fp8bq_gemm_mxfp4", GEMM), ("fp8bq_grouped_gemm_mxfp4", GROUPED),
                                   ("fp8bq_grouped_wgrad_mxfp4", GROUPED)])
def test_product_refusals(L, fn, ok):
    d = len(ok) - len(GEMM)
    p = lambda i: f"a{i + d}"                   # noqa: E731
    for i in (0, 1, 2):
        expect(L, fb.E_INVAL, fn, ok, **{p(i): 0})
        expect(L, fb.E_INVAL, fn, ok, **{p(i): -5})
        expect(L, fb.E_SHAPE, fn, ok, **{p(i): BIG, p(4): BIG, p(6): BIG, p(8): BIG, p(10): BIG, p(13): BIG})
    for i in (3, 5, 7, 9, 11):
        expect(L, fb.E_INVAL, fn, ok, **{p(i): None})
    expect(L, fb.E_INVAL, fn, ok, **{p(4): 240})
    expect(L, fb.E_INVAL, fn, ok, **{p(8): 128})
    expect(L, fb.E_INVAL, fn, ok, **{p(6): 69})
    expect(L, fb.E_INVAL, fn, ok, **{p(10): 89})
    expect(L, fb.E_INVAL, fn, ok, **{p(12): 1})
    expect(L, fb.E_INVAL, fn, ok, **{p(13): 89})
    expect(L, fb.E_ALIGN, fn, ok, **{p(3): A16 + 8})
    expect(L, fb.E_ALIGN, fn, ok, **{p(8): 264})
    expect(L, fb.E_ALIGN, fn, ok, **{p(9): S8 + 4})
    expect(L, fb.E_ALIGN, fn, ok, **{p(11): A16 + 1})
    expect(L, fb.E_SHAPE, fn, ok, **{p(4): 1 << 24})
    if d:
        expect(L, fb.E_INVAL, fn, ok, a1=None)
        expect(L, fb.E_ALIGN, fn, ok, a1=O4 + 2)
        for g in (0, -1, 257):
            expect(L, fb.E_SHAPE, fn, ok, a0=g)


def test_plan_refusals(L):
    fn = "fp8bq_moe_plan"
    for i in (0, 6, 7, 8, 10, 11):
        expect(L, fb.E_INVAL, fn, PLAN, **{f"a{i}": None})
        expect(L, fb.E_ALIGN, fn, PLAN, **{f"a{i}": O4 + 1})
    expect(L, fb.E_INVAL, fn, PLAN, a1=0)
    expect(L, fb.E_INVAL, fn, PLAN, a2=-1)
    expect(L, fb.E_INVAL, fn, PLAN, a3=7)
    for pad in (0, 1025):
        expect(L, fb.E_INVAL, fn, PLAN, a5=pad)
    for g in (0, 257):
        expect(L, fb.E_SHAPE, fn, PLAN, a4=g)
    expect(L, fb.E_INVAL, fn, PLAN, a9=800 + 16 * 31 - 1)
    expect(L, fb.E_SHAPE, fn, PLAN, a1=BIG)
    expect(L, fb.E_SHAPE, fn, PLAN, a1=1 << 29, a9=BIG)
    expect(L, fb.E_SHAPE, fn, PLAN, a9=1 << 30)


@pytest.mark.parametrize("fn,ok", [("fp8bq_moe_balance", BALANCE), ("fp8bq_moe_balance_grad", GRAD)])
def test_balance_refusals(L, fn, ok):
    d = 1 if "grad" in fn else 0
    p = lambda i: f"a{i + d}"                   # noqa: E731
    pointers = (0, 5, 12, 13, 14, 15) if not d else (-1, 0, 5, 12, 13, 14)
    for i in pointers:
        expect(L, fb.E_INVAL, fn, ok, **{p(i): None})
        expect(L, fb.E_ALIGN, fn, ok, **{p(i): O4 + 1})
    expect(L, fb.E_INVAL, fn, ok, **{p(1): 9})
    for i in (2, 3, 6, 9):
        expect(L, fb.E_INVAL, fn, ok, **{p(i): 0})
    expect(L, fb.E_INVAL, fn, ok, **{p(4): 63})
    expect(L, fb.E_INVAL, fn, ok, **{p(7): 5})
    expect(L, fb.E_INVAL, fn, ok, **{p(8): None})
    expect(L, fb.E_INVAL, fn, ok, **{p(10): 2})
    expect(L, fb.E_SHAPE, fn, ok, **{p(3): 1025, p(4): 1025})
    expect(L, fb.E_SHAPE, fn, ok, **{p(9): 65535})
    expect(L, fb.E_SHAPE, fn, ok, **{p(2): BIG})
    expect(L, fb.E_SHAPE, fn, ok, **{p(4): BIG})
    expect(L, fb.E_SHAPE, fn, ok, **{p(2): 1 << 21, p(6): 1 << 10, p(7): 1 << 10})   # an expert's count past int32
    expect(L, fb.E_SHAPE, fn, ok, **{p(6): BIG, p(7): BIG})
    if d:
        expect(L, fb.E_INVAL, fn, ok, a16=63)


def test_balance_workspace_size(L):
    n = ctypes.c_int64(-1)
    assert L.fp8bq_moe_balance_workspace_size(16384, 256, 4, ctypes.byref(n)) == fb.OK and n.value > 0
    assert fb.fp8bq_moe_balance_workspace_size(1, 1, 1) >= 4 * 5
    assert L.fp8bq_moe_balance_workspace_size(1, 1, 1, None) == fb.E_INVAL
    assert L.fp8bq_moe_balance_workspace_size(0, 1, 1, ctypes.byref(n)) == fb.E_INVAL
    assert L.fp8bq_moe_balance_workspace_size(1, 2000, 1, ctypes.byref(n)) == fb.E_SHAPE


def test_good_arguments_reach_the_device_check(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible; valid arguments would launch")
    for fn, ok in (("fp8bq_quant_mxfp4_1x32", QUANT), ("fp8bq_dispatch_mxfp4_1x32", DISPATCH),
                   ("fp8bq_dequant_mxfp4_1x32", DEQUANT), ("fp8bq_gemm_mxfp4", GEMM),
                   ("fp8bq_grouped_gemm_mxfp4", GROUPED), ("fp8bq_grouped_wgrad_mxfp4", GROUPED),
                   ("fp8bq_moe_plan", PLAN), ("fp8bq_moe_balance", BALANCE), ("fp8bq_moe_balance_grad", GRAD)):
        expect(L, fb.E_DEVICE, fn, ok)


def test_tensor_layer_refusals():
    """What the C entry cannot see (types, shapes, strides, places) raises ValueError."""
    import torch
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((1, 4, 8), dtype=torch.uint8)
    off = torch.zeros(3, dtype=torch.int32)
    idx = torch.zeros((4, 2), dtype=torch.int32)
    logits = torch.zeros((4, 8))
    bq, bs = q.expand(2, 4, 128).contiguous(), s.expand(2, 1, 4, 8).contiguous()
    bad = [
        lambda: fb.quant_mxfp4_1x32(x),                                        # not on a GPU
        lambda: fb.quant_mxfp4_1x32(x.double()),
        lambda: fb.quant_mxfp4_1x32(x.t()),
        lambda: fb.quant_mxfp4_1x32(x[0]),
        lambda: fb.quant_mxfp4_1x32(x[:0]),
        lambda: fb.quant_mxfp4_1x32(x, rowwise=False),
        lambda: fb.dispatch_mxfp4_1x32(x, off.long()),
        lambda: fb.dispatch_mxfp4_1x32(x, off[::2]),
        lambda: fb.dispatch_mxfp4_1x32(x, off[:0]),
        lambda: fb.dequant_mxfp4_1x32(q, s, 257),
        lambda: fb.dequant_mxfp4_1x32(q, s, 0),
        lambda: fb.dequant_mxfp4_1x32(q, s, 64, torch.int8),
        lambda: fb.gemm_mxfp4(q, s, q[:, :64], s),
        lambda: fb.gemm_mxfp4(q, s[:, :3], q, s),
        lambda: fb.gemm_mxfp4(q, s, torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((2, 4, 8), dtype=torch.uint8)),
        lambda: fb.gemm_mxfp4(q.int(), s, q, s),
        lambda: fb.gemm_mxfp4(q, s, q, s),
        lambda: fb.grouped_gemm_mxfp4(off.long(), q, s, bq, bs),
        lambda: fb.grouped_gemm_mxfp4(off[:2], q, s, bq, bs),
        lambda: fb.grouped_gemm_mxfp4(off, q, s, bq, s),
        lambda: fb.grouped_gemm_mxfp4(off, q, s, bq.transpose(0, 1), bs),
        lambda: fb.grouped_wgrad_mxfp4(off[:1], q, s, q, s),
        lambda: fb.moe_plan(idx.long(), 4),
        lambda: fb.moe_plan(idx, 0),
        lambda: fb.moe_plan(idx[0], 4),
        lambda: fb.moe_balance(logits, idx, 1.0, "tanh"),
        lambda: fb.moe_balance(logits, idx[:3], 1.0),
        lambda: fb.moe_balance(logits.int(), idx, 1.0),
        lambda: fb.moe_balance(logits, idx, 1.0, seq_off=off[:1]),
        lambda: fb.moe_balance(logits, idx, 1.0, seq_off=off.long()),
        lambda: fb.moe_balance_grad(torch.zeros(()), logits, idx, torch.zeros((2, 8), dtype=torch.int32),
                                    torch.zeros(1, dtype=torch.int32), 1.0),
        lambda: fb.moe_balance_grad(torch.zeros(2), logits, idx, torch.zeros((1, 8), dtype=torch.int32),
                                    torch.zeros(1, dtype=torch.int32), 1.0),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("accepted:", i)


def test_message_of_a_refusal():
    with pytest.raises(fb.Fp8bqError, match="E_INVAL.*no output"):
        fb.fp8bq_quant_mxfp4_1x32(A16, 0, 4, 64, 64, None, 0, None, 0, None, 0, None, 0)
