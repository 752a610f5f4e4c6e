"""fp8bq: fine-grained FP8 (E4M3, 1x128 / 128x128) quantisation and block-scaled
FP8 GEMM for AMD MI355X (gfx950).

Thin ctypes binding over the C ABI in include/fp8bq.h (libfp8bq.so, built in
this package directory by `build.py`). Every step of the computation runs in
the library's HIP kernels; this module only marshals arguments. There is no
fallback: if the library is missing or the device is not gfx950, calls raise.

Two layers with the C names:

* `fp8bq_quant_act_1x128`, `fp8bq_quant_w_128x128`, `fp8bq_requant_t_128x1`,
  `fp8bq_gemm`, `fp8bq_gemm_quant`, `fp8bq_grouped_gemm`,
  `fp8bq_grouped_gemm_decode`, `fp8bq_grouped_gemm_decode_workspace_size`,
  `fp8bq_grouped_gemm_decode_ws`, `fp8bq_grouped_gemm_decode_noalloc`, `fp8bq_cache_e5m6_1x128`,
  `fp8bq_uncache_e5m6_1x128`, `fp8bq_requant_e5m6_t_128x1`, `fp8bq_quant_mxfp4_1x32`,
  `fp8bq_dispatch_mxfp4_1x32`, `fp8bq_dequant_mxfp4_1x32`, `fp8bq_gemm_mxfp4`,
  `fp8bq_grouped_gemm_mxfp4`, `fp8bq_grouped_wgrad_mxfp4`, `fp8bq_moe_plan`, `fp8bq_moe_balance`,
  `fp8bq_moe_balance_workspace_size`, `fp8bq_moe_balance_grad`: pointer-level, exactly the C signatures (ints
  for pointers and the stream); a non-zero status raises `Fp8bqError`.
* `quant_act_1x128`, `quant_w_128x128`, `requant_t_128x1`, `gemm`,
  `gemm_quant`, `grouped_gemm`, `grouped_gemm_decode`, `cache_e5m6_1x128`,
  `uncache_e5m6_1x128`, `requant_e5m6_t_128x1`, and the MXFP4 and routing operators
  (`quant_mxfp4_1x32`, `dispatch_mxfp4_1x32`, `dequant_mxfp4_1x32`, `gemm_mxfp4`,
  `grouped_gemm_mxfp4`, `grouped_wgrad_mxfp4`, `moe_plan`, `moe_balance`, `moe_balance_grad`): take torch tensors on
  the GPU, allocate the outputs with torch (memory and streams are the only
  things torch provides) and call the same entry points on the current stream.
"""

from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8bq.so")

OK, E_INVAL, E_SHAPE, E_ALIGN, E_DEVICE, E_HIP = range(6)
STATUS_NAMES = {0: "OK", 1: "E_INVAL", 2: "E_SHAPE", 3: "E_ALIGN", 4: "E_DEVICE", 5: "E_HIP"}
FPROP, DGRAD, WGRAD = 0, 1, 2
ACT_ROWWISE, ACT_COLWISE = 0, 1
BF16, FP16, FP32 = 0, 1, 2
MX_NOSAT = 0x20     # MXFP4 scales that never saturate an element
SOFTMAX, SIGMOID = 0, 1
MOE_PLAN_WORKSPACE_BYTES = 256 * 256 * 4
SCALE_POW2 = 0x10   # power-of-two scales (OR into the act mode / gemm op; `flags` elsewhere)

EXPORTS = ("fp8bq_quant_act_1x128", "fp8bq_quant_w_128x128", "fp8bq_requant_t_128x1", "fp8bq_gemm",
           "fp8bq_gemm_quant", "fp8bq_grouped_gemm", "fp8bq_grouped_gemm_decode",
           "fp8bq_grouped_gemm_decode_workspace_size", "fp8bq_grouped_gemm_decode_ws",
           "fp8bq_grouped_gemm_decode_noalloc", "fp8bq_cache_e5m6_1x128",
           "fp8bq_uncache_e5m6_1x128", "fp8bq_requant_e5m6_t_128x1", "fp8bq_quant_mxfp4_1x32",
           "fp8bq_dispatch_mxfp4_1x32", "fp8bq_dequant_mxfp4_1x32", "fp8bq_gemm_mxfp4", "fp8bq_grouped_gemm_mxfp4",
           "fp8bq_grouped_wgrad_mxfp4", "fp8bq_moe_plan", "fp8bq_moe_balance_workspace_size", "fp8bq_moe_balance",
           "fp8bq_moe_balance_grad", "fp8bq_last_error", "fp8bq_version")


class Fp8bqError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libfp8bq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m fp8_fine_grained_fp8bq_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, fp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
        L.fp8bq_quant_act_1x128.argtypes = [vp, i64, i64, i64, i32, vp, i64, fp, i64, vp]
        L.fp8bq_quant_w_128x128.argtypes = [vp, i64, i64, i64, vp, i64, fp, i64, vp, i64, i32, vp]
        L.fp8bq_requant_t_128x1.argtypes = [vp, i64, i64, i64, fp, i64, vp, i64, fp, i64, i32, vp]
        L.fp8bq_cache_e5m6_1x128.argtypes = [vp, i64, i64, i64, vp, i64, fp, i64, vp]
        L.fp8bq_uncache_e5m6_1x128.argtypes = [vp, i64, i64, i64, fp, i64, vp, i64, vp]
        L.fp8bq_requant_e5m6_t_128x1.argtypes = [vp, i64, i64, i64, fp, i64, vp, i64, fp, i64, vp]
        L.fp8bq_gemm.argtypes = [i32, i64, i64, i64, vp, i64, fp, i64, vp, i64, fp, i64, vp, i64, vp]
        L.fp8bq_gemm_quant.argtypes = [i32, i64, i64, i64, vp, i64, fp, i64, vp, i64, fp, i64, vp, i64,
                                       vp, i64, fp, i64, i32, vp]
        L.fp8bq_grouped_gemm.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_int64), i64, i64,
                                         vp, i64, fp, i64, vp, i64, fp, i64, vp, i64, i32, vp]
        for f in ("fp8bq_quant_act_1x128", "fp8bq_quant_w_128x128", "fp8bq_requant_t_128x1", "fp8bq_gemm",
                  "fp8bq_grouped_gemm", "fp8bq_cache_e5m6_1x128", "fp8bq_uncache_e5m6_1x128",
                  "fp8bq_requant_e5m6_t_128x1"):
            getattr(L, f).restype = ctypes.c_int
        L.fp8bq_last_error.restype = ctypes.c_char_p
        L.fp8bq_grouped_gemm_decode.argtypes = L.fp8bq_grouped_gemm.argtypes
        L.fp8bq_grouped_gemm_decode_workspace_size.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_int64), i64,
                                                               i64, ctypes.POINTER(ctypes.c_int64)]
        L.fp8bq_grouped_gemm_decode_workspace_size.restype = ctypes.c_int
        L.fp8bq_grouped_gemm_decode_ws.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_int64), i64, i64,
                                                   vp, i64, fp, i64, vp, i64, fp, i64, vp, i64, vp, i64, i32, vp]
        L.fp8bq_grouped_gemm_decode_ws.restype = ctypes.c_int
        L.fp8bq_grouped_gemm_decode_noalloc.argtypes = L.fp8bq_grouped_gemm.argtypes
        L.fp8bq_grouped_gemm_decode_noalloc.restype = ctypes.c_int
        mx = [vp, i64, vp, i64]                 # codes, ld, scales, ld
        L.fp8bq_quant_mxfp4_1x32.argtypes = [vp, i32, i64, i64, i64, *mx, *mx, i32, vp]
        L.fp8bq_dispatch_mxfp4_1x32.argtypes = [vp, i32, i64, i64, i64, vp, i64, *mx, *mx, i32, vp]
        L.fp8bq_dequant_mxfp4_1x32.argtypes = [vp, i64, i64, i64, vp, i64, vp, i32, i64, vp]
        L.fp8bq_gemm_mxfp4.argtypes = [i64, i64, i64, *mx, *mx, vp, i32, i64, vp]
        L.fp8bq_grouped_gemm_mxfp4.argtypes = [ctypes.c_int32, vp, i64, i64, i64, *mx, *mx, vp, i32, i64, vp]
        L.fp8bq_grouped_wgrad_mxfp4.argtypes = L.fp8bq_grouped_gemm_mxfp4.argtypes
        L.fp8bq_moe_plan.argtypes = [vp, i64, i64, i64, ctypes.c_int32, i64, vp, vp, vp, i64, vp, vp, vp]
        L.fp8bq_moe_balance_workspace_size.argtypes = [i64, i64, i64, ctypes.POINTER(ctypes.c_int64)]
        routing = [vp, i32, i64, i64, i64, vp, i64, i64, vp, i64, i32, ctypes.c_float]   # logits .. coef
        L.fp8bq_moe_balance.argtypes = [*routing, vp, vp, vp, vp, vp]
        L.fp8bq_moe_balance_grad.argtypes = [vp, *routing, vp, vp, vp, i64, vp]
        for f in EXPORTS:
            if "mxfp4" in f or "moe" in f:
                getattr(L, f).restype = ctypes.c_int
        L.fp8bq_last_error.argtypes = []
        L.fp8bq_version.restype = ctypes.c_char_p
        L.fp8bq_version.argtypes = []
        _lib = L
    return _lib


def _check(fn: str, status: int) -> int:
    if status != OK:
        raise Fp8bqError(fn, status, lib().fp8bq_last_error().decode())
    return status


# ---------------------------------------------------------------------------
# pointer-level entry points (C names)
# ---------------------------------------------------------------------------

def fp8bq_quant_act_1x128(x, rows, cols, ldx, mode, q, ldq, s, lds, stream=0):
    return _check("fp8bq_quant_act_1x128",
                  lib().fp8bq_quant_act_1x128(x, rows, cols, ldx, mode, q, ldq, s, lds, stream))


def fp8bq_quant_w_128x128(w, n, k, ldw, q, ldq, s, lds, qt, ldqt, flags=0, stream=0):
    return _check("fp8bq_quant_w_128x128",
                  lib().fp8bq_quant_w_128x128(w, n, k, ldw, q, ldq, s, lds, qt, ldqt, flags, stream))


def fp8bq_requant_t_128x1(q, rows, cols, ldq, s, lds, qt, ldqt, st, ldst, flags=0, stream=0):
    return _check("fp8bq_requant_t_128x1",
                  lib().fp8bq_requant_t_128x1(q, rows, cols, ldq, s, lds, qt, ldqt, st, ldst, flags, stream))


def fp8bq_gemm(op, m, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, ldo, stream=0):
    return _check("fp8bq_gemm",
                  lib().fp8bq_gemm(op, m, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, ldo, stream))


def fp8bq_gemm_quant(op, m, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, ldo, q, ldq, s, lds, qflags=0,
                     stream=0):
    return _check("fp8bq_gemm_quant",
                  lib().fp8bq_gemm_quant(op, m, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, ldo, q, ldq, s, lds,
                                         qflags, stream))


def fp8bq_grouped_gemm(groups, row_off, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, ldo, flags=0,
                       stream=0):
    """`row_off` is a sequence of groups + 1 ints (host memory)."""
    arr = (ctypes.c_int64 * (groups + 1))(*[int(v) for v in row_off]) if row_off is not None else None
    return _check("fp8bq_grouped_gemm",
                  lib().fp8bq_grouped_gemm(groups, arr, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb,
                                           out, ldo, flags, stream))


def fp8bq_grouped_gemm_decode(groups, row_off, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, ldo, flags=0,
                              stream=0):
    """`row_off` is a sequence of groups + 1 ints (host memory), any counts up to 256 per group."""
    arr = (ctypes.c_int64 * (groups + 1))(*[int(v) for v in row_off]) if row_off is not None else None
    return _check("fp8bq_grouped_gemm_decode",
                  lib().fp8bq_grouped_gemm_decode(groups, arr, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb,
                                                  out, ldo, flags, stream))


def version() -> str:
    return lib().fp8bq_version().decode()


# ---------------------------------------------------------------------------
# torch-tensor convenience layer (allocation + marshalling only)
# ---------------------------------------------------------------------------

def _stream(t):
    import torch
    return torch.cuda.current_stream(t.device).cuda_stream


def _bf16_2d(t, name):
    import torch
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D row-major bf16 tensor (got {t.dtype}, {tuple(t.shape)})")
    return t


def quant_act_1x128(x, mode: int = ACT_ROWWISE):
    """x bf16 [rows, cols] -> (q uint8, s float32) as laid out by the C ABI:
    ROWWISE q [rows, cols], s [cols/128, rows]; COLWISE q [cols, rows], s [rows/128, cols].
    `mode` may include SCALE_POW2 (power-of-two scales)."""
    import torch
    _bf16_2d(x, "x")
    rows, cols = x.shape
    if (mode & ~SCALE_POW2) == ACT_ROWWISE:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
        s = torch.empty((cols // 128, rows), dtype=torch.float32, device=x.device)
        ldq, lds = cols, rows
    else:
        q = torch.empty((cols, rows), dtype=torch.uint8, device=x.device)
        s = torch.empty((rows // 128, cols), dtype=torch.float32, device=x.device)
        ldq, lds = rows, cols
    fp8bq_quant_act_1x128(x.data_ptr(), rows, cols, x.stride(0), mode, q.data_ptr(), ldq,
                          s.data_ptr(), lds, _stream(x))
    return q, s


def quant_w_128x128(w, transposed_copy: bool = False, pow2: bool = False):
    """w bf16 [n, k] -> (q uint8 [n, k], s float32 [n/128, k/128], qt uint8 [k, n] or None);
    pow2 selects power-of-two scales."""
    import torch
    _bf16_2d(w, "w")
    n, k = w.shape
    q = torch.empty((n, k), dtype=torch.uint8, device=w.device)
    s = torch.empty((n // 128, k // 128), dtype=torch.float32, device=w.device)
    qt = torch.empty((k, n), dtype=torch.uint8, device=w.device) if transposed_copy else None
    fp8bq_quant_w_128x128(w.data_ptr(), n, k, w.stride(0), q.data_ptr(), k, s.data_ptr(), k // 128,
                          qt.data_ptr() if qt is not None else None, n, SCALE_POW2 if pow2 else 0, _stream(w))
    return q, s, qt


def fp8bq_cache_e5m6_1x128(x, rows, cols, ldx, q, ldq, s, lds, stream=0):
    return _check("fp8bq_cache_e5m6_1x128", lib().fp8bq_cache_e5m6_1x128(x, rows, cols, ldx, q, ldq, s, lds, stream))


def fp8bq_uncache_e5m6_1x128(q, rows, cols, ldq, s, lds, y, ldy, stream=0):
    return _check("fp8bq_uncache_e5m6_1x128",
                  lib().fp8bq_uncache_e5m6_1x128(q, rows, cols, ldq, s, lds, y, ldy, stream))


def fp8bq_requant_e5m6_t_128x1(q, rows, cols, ldq, s, lds, qt, ldqt, st, ldst, stream=0):
    return _check("fp8bq_requant_e5m6_t_128x1",
                  lib().fp8bq_requant_e5m6_t_128x1(q, rows, cols, ldq, s, lds, qt, ldqt, st, ldst, stream))


def cache_e5m6_1x128(x):
    """bf16 [rows, cols] (int16/bfloat16 storage) -> (q uint8 [rows, 1.5 cols]: packed 12-bit E5M6
    codes, s float32 [cols/128, rows]: chunk-major power-of-two 1x128 tile scales)."""
    import torch
    if x.dim() != 2 or x.element_size() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D row-major 16-bit tensor of bf16 patterns")
    rows, cols = x.shape
    ldq = (cols * 3 // 2 + 15) // 16 * 16
    q = torch.empty((rows, ldq), dtype=torch.uint8, device=x.device)
    s = torch.empty((cols // 128, rows), dtype=torch.float32, device=x.device)
    fp8bq_cache_e5m6_1x128(x.data_ptr(), rows, cols, x.stride(0), q.data_ptr(), ldq, s.data_ptr(), rows, _stream(x))
    return q[:, : cols * 3 // 2], s


def uncache_e5m6_1x128(q, s, cols):
    """Packed E5M6 codes q (rows of >= 1.5 cols bytes, row stride q.stride(0)) and their scales s
    [cols/128, >=rows] -> bf16 [rows, cols] (torch.bfloat16)."""
    import torch
    if q.dtype != torch.uint8 or q.dim() != 2 or q.stride(1) != 1:
        raise ValueError("q must be a 2-D row-major uint8 tensor")
    rows = q.shape[0]
    y = torch.empty((rows, cols), dtype=torch.bfloat16, device=q.device)
    fp8bq_uncache_e5m6_1x128(q.data_ptr(), rows, cols, q.stride(0), s.data_ptr(), s.stride(0), y.data_ptr(), cols,
                             _stream(q))
    return y


def requant_e5m6_t_128x1(q, s, cols):
    """E5M6 cache q (rows of >= 1.5 cols bytes, row stride q.stride(0)) with its power-of-two
    scales s [cols/128, >=rows] -> (qt uint8 [cols, rows], st float32 [rows/128, cols]): the cached
    values re-quantised to E4M3 in 128x1 tiles with power-of-two scales, COLWISE layout."""
    import torch
    if q.dtype != torch.uint8 or q.dim() != 2 or q.stride(1) != 1:
        raise ValueError("q must be a 2-D row-major uint8 tensor")
    if s.dtype != torch.float32 or s.dim() != 2 or s.stride(1) != 1:
        raise ValueError("s must be a 2-D row-major float32 tensor")
    rows = q.shape[0]
    qt = torch.empty((cols, rows), dtype=torch.uint8, device=q.device)
    st = torch.empty((rows // 128, cols), dtype=torch.float32, device=q.device)
    fp8bq_requant_e5m6_t_128x1(q.data_ptr(), rows, cols, q.stride(0), s.data_ptr(), s.stride(0), qt.data_ptr(),
                               rows, st.data_ptr(), cols, _stream(q))
    return qt, st


def requant_t_128x1(q, s, pow2_scales=False):
    """FP8 activation cache q uint8 [rows, cols] with chunk-major 1x128 scales s [cols/128, >=rows]
    -> (qt uint8 [cols, rows], st float32 [rows/128, cols]): 128x1 tiles with power-of-two scales,
    the layout of COLWISE quantisation. pow2_scales: s holds powers of two (the kernel for that
    case; the result is the same)."""
    import torch
    if q.dtype != torch.uint8 or q.dim() != 2 or q.stride(1) != 1:
        raise ValueError("q must be a 2-D row-major uint8 tensor")
    if s.dtype != torch.float32 or s.dim() != 2 or s.stride(1) != 1:
        raise ValueError("s must be a 2-D row-major float32 tensor")
    rows, cols = q.shape
    qt = torch.empty((cols, rows), dtype=torch.uint8, device=q.device)
    st = torch.empty((rows // 128, cols), dtype=torch.float32, device=q.device)
    fp8bq_requant_t_128x1(q.data_ptr(), rows, cols, q.stride(0), s.data_ptr(), s.stride(0), qt.data_ptr(), rows,
                          st.data_ptr(), cols, SCALE_POW2 if pow2_scales else 0, _stream(q))
    return qt, st


def gemm(op: int, a, sa, b, sb, out=None):
    """a uint8 [m, k] with chunk-major scales sa [k/128, >=m]; b uint8 [n, k] with
    sb laid out per `op` (see include/fp8bq.h); `op` may include SCALE_POW2. Returns out
    (bf16 or fp32) [m, n]."""
    import torch
    m, k = a.shape
    n = b.shape[0]
    if out is None:
        dt = torch.float32 if (op & ~SCALE_POW2) == WGRAD else torch.bfloat16
        out = torch.empty((m, n), dtype=dt, device=a.device)
    fp8bq_gemm(op, m, n, k, a.data_ptr(), a.stride(0), sa.data_ptr(), sa.stride(0),
               b.data_ptr(), b.stride(0), sb.data_ptr(), sb.stride(0), out.data_ptr(), out.stride(0),
               _stream(a))
    return out


def gemm_quant(op: int, a, sa, b, sb, with_out: bool = True, qpow2: bool = False):
    """fp8bq_gemm (FPROP / DGRAD, `op` may include SCALE_POW2) that also quantises its bf16
    output in 1x128 tiles. Returns (out bf16 [m, n] or None, q uint8 [m, n], s float32
    [n/128, m]); qpow2 selects power-of-two output scales."""
    import torch
    m, k = a.shape
    n = b.shape[0]
    out = torch.empty((m, n), dtype=torch.bfloat16, device=a.device) if with_out else None
    q = torch.empty((m, n), dtype=torch.uint8, device=a.device)
    s = torch.empty((n // 128, m), dtype=torch.float32, device=a.device)
    fp8bq_gemm_quant(op, m, n, k, a.data_ptr(), a.stride(0), sa.data_ptr(), sa.stride(0),
                     b.data_ptr(), b.stride(0), sb.data_ptr(), sb.stride(0),
                     out.data_ptr() if out is not None else None, n, q.data_ptr(), n, s.data_ptr(), m,
                     SCALE_POW2 if qpow2 else 0, _stream(a))
    return out, q, s


def grouped_gemm(row_off, a, sa, b, sb, out=None, pow2: bool = False):
    """row_off: host sequence of G + 1 row offsets (multiples of 128); a uint8 [m, k];
    sa [k/128, >=m]; b uint8 [G, n, k]; sb float32 [G, n/128, k/128]. Returns bf16 [m, n].
    pow2: power-of-two scales applied by the matrix instruction."""
    import torch
    G, n, k = b.shape
    m = a.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    fp8bq_grouped_gemm(G, list(row_off), n, k, a.data_ptr(), a.stride(0), sa.data_ptr(), sa.stride(0),
                       b.data_ptr(), b.stride(1), sb.data_ptr(), sb.stride(1), out.data_ptr(),
                       out.stride(0), SCALE_POW2 if pow2 else 0, _stream(a))
    return out


def _offsets(groups, row_off):
    return (ctypes.c_int64 * (groups + 1))(*[int(v) for v in row_off]) if row_off is not None else None


def fp8bq_grouped_gemm_decode_workspace_size(groups, row_off, n, k):
    """Bytes of workspace fp8bq_grouped_gemm_decode_ws needs (row_off: host sequence)."""
    out = ctypes.c_int64(-1)
    _check("fp8bq_grouped_gemm_decode_workspace_size",
           lib().fp8bq_grouped_gemm_decode_workspace_size(groups, _offsets(groups, row_off), n, k, ctypes.byref(out)))
    return out.value


def fp8bq_grouped_gemm_decode_ws(groups, row_off, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, ldo, workspace,
                                 workspace_bytes, flags=0, stream=0):
    return _check("fp8bq_grouped_gemm_decode_ws",
                  lib().fp8bq_grouped_gemm_decode_ws(groups, _offsets(groups, row_off), n, k, a, lda, sa, ldsa, b,
                                                     ldb, sb, ldsb, out, ldo, workspace, workspace_bytes, flags,
                                                     stream))


def fp8bq_grouped_gemm_decode_noalloc(groups, row_off, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, ldo, flags=0,
                                      stream=0):
    return _check("fp8bq_grouped_gemm_decode_noalloc",
                  lib().fp8bq_grouped_gemm_decode_noalloc(groups, _offsets(groups, row_off), n, k, a, lda, sa, ldsa, b,
                                                          ldb, sb, ldsb, out, ldo, flags, stream))


DECODE_NOALLOC_SCRATCH_BYTES = 32 << 20

_workspaces = {}


def decode_workspace(nbytes, device):
    """A zero-filled device workspace of at least nbytes for fp8bq_grouped_gemm_decode_ws, kept
    per device and reused (every call leaves its counters zero). Calls that share it must run
    on one stream."""
    import torch
    key = torch.device(device).index if torch.device(device).index is not None else torch.cuda.current_device()
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def grouped_gemm_decode(row_off, a, sa, b, sb, out=None, split=True):
    """Decode-shape grouped Fprop: row_off host sequence of G + 1 offsets (any counts up to
    256 rows per expert); a uint8 [m, k]; sa [k/128, >=m]; b uint8 [G, n, k];
    sb float32 [G, n/128, k/128]. Returns bf16 [m, n]. split: experts of more than 32 rows
    run as 128-column half-K workgroup pairs through a cached workspace."""
    import torch
    G, n, k = b.shape
    m = a.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    if split:
        need = fp8bq_grouped_gemm_decode_workspace_size(G, list(row_off), n, k)
        ws = decode_workspace(need, a.device) if need > 0 else None
        fp8bq_grouped_gemm_decode_ws(G, list(row_off), n, k, a.data_ptr(), a.stride(0), sa.data_ptr(), sa.stride(0),
                                     b.data_ptr(), b.stride(1), sb.data_ptr(), sb.stride(1), out.data_ptr(),
                                     out.stride(0), ws.data_ptr() if ws is not None else None,
                                     ws.numel() if ws is not None else 0, 0, _stream(a))
        return out
    fp8bq_grouped_gemm_decode(G, list(row_off), n, k, a.data_ptr(), a.stride(0), sa.data_ptr(), sa.stride(0),
                              b.data_ptr(), b.stride(1), sb.data_ptr(), sb.stride(1), out.data_ptr(),
                              out.stride(0), 0, _stream(a))
    return out


# ---------------------------------------------------------------------------
# MXFP4 operators and the routing of tokens to experts: pointer level
# ---------------------------------------------------------------------------

def fp8bq_quant_mxfp4_1x32(x, xtype, rows, cols, ldx, q, ldq, s, lds, qt, ldqt, st, ldst, flags=0, stream=0):
    return _check("fp8bq_quant_mxfp4_1x32", lib().fp8bq_quant_mxfp4_1x32(x, xtype, rows, cols, ldx, q, ldq, s, lds, qt,
                                                                         ldqt, st, ldst, flags, stream))


def fp8bq_dispatch_mxfp4_1x32(x, xtype, xrows, cols, ldx, src, rows, q, ldq, s, lds, qt, ldqt, st, ldst, flags=0,
                              stream=0):
    return _check("fp8bq_dispatch_mxfp4_1x32",
                  lib().fp8bq_dispatch_mxfp4_1x32(x, xtype, xrows, cols, ldx, src, rows, q, ldq, s, lds, qt, ldqt, st,
                                                  ldst, flags, stream))


def fp8bq_dequant_mxfp4_1x32(q, rows, cols, ldq, s, lds, y, ytype, ldy, stream=0):
    return _check("fp8bq_dequant_mxfp4_1x32",
                  lib().fp8bq_dequant_mxfp4_1x32(q, rows, cols, ldq, s, lds, y, ytype, ldy, stream))


def fp8bq_gemm_mxfp4(m, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, otype, ldo, stream=0):
    return _check("fp8bq_gemm_mxfp4",
                  lib().fp8bq_gemm_mxfp4(m, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, otype, ldo, stream))


def fp8bq_grouped_gemm_mxfp4(groups, row_off, m, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, otype, ldo, stream=0):
    """`row_off` is a device pointer (int32, groups + 1), unlike fp8bq_grouped_gemm's."""
    return _check("fp8bq_grouped_gemm_mxfp4",
                  lib().fp8bq_grouped_gemm_mxfp4(groups, row_off, m, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out,
                                                 otype, ldo, stream))


def fp8bq_grouped_wgrad_mxfp4(groups, row_off, m, n, rows, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, otype, ldo,
                              stream=0):
    return _check("fp8bq_grouped_wgrad_mxfp4",
                  lib().fp8bq_grouped_wgrad_mxfp4(groups, row_off, m, n, rows, a, lda, sa, ldsa, b, ldb, sb, ldsb, out,
                                                  otype, ldo, stream))


def fp8bq_moe_plan(idx, tokens, topk, ldidx, groups, pad, counts, row_off, src, cap, pos, workspace, stream=0):
    return _check("fp8bq_moe_plan", lib().fp8bq_moe_plan(idx, tokens, topk, ldidx, groups, pad, counts, row_off, src,
                                                         cap, pos, workspace, stream))


def fp8bq_moe_balance_workspace_size(tokens, experts, sequences):
    """Bytes of workspace fp8bq_moe_balance needs."""
    out = ctypes.c_int64(-1)
    _check("fp8bq_moe_balance_workspace_size",
           lib().fp8bq_moe_balance_workspace_size(tokens, experts, sequences, ctypes.byref(out)))
    return out.value


def fp8bq_moe_balance(logits, ltype, tokens, experts, ldl, idx, topk, ldidx, seq_off, sequences, score, coef, loss,
                      counts, real, workspace, stream=0):
    return _check("fp8bq_moe_balance",
                  lib().fp8bq_moe_balance(logits, ltype, tokens, experts, ldl, idx, topk, ldidx, seq_off, sequences,
                                          score, coef, loss, counts, real, workspace, stream))


def fp8bq_moe_balance_grad(dloss, logits, ltype, tokens, experts, ldl, idx, topk, ldidx, seq_off, sequences, score,
                           coef, counts, real, dlogits, lddl, stream=0):
    return _check("fp8bq_moe_balance_grad",
                  lib().fp8bq_moe_balance_grad(dloss, logits, ltype, tokens, experts, ldl, idx, topk, ldidx, seq_off,
                                               sequences, score, coef, counts, real, dlogits, lddl, stream))


# ---------------------------------------------------------------------------
# the same on torch tensors
# ---------------------------------------------------------------------------
# These calls run on the tensors' device (also when it is not the current one)
# and on that device's current stream; every tensor of a call is on one device.

def _on(*tensors):
    """The one device of the tensors, made current for the call."""
    import torch
    dev = tensors[0].device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {t.device}")
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on the GPU, got {dev}")
    return torch.cuda.device(dev)


def _dtype(t, name):
    import torch
    code = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}.get(t.dtype if hasattr(t, "dtype") else t)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32 (got {t.dtype if hasattr(t, 'dtype') else t})")
    return code


def _matrix(t, name):
    if t.dim() != 2 or t.shape[0] < 1 or t.shape[1] < 1 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be a non-empty 2-D row-major tensor (got {tuple(t.shape)}, strides {t.stride()})")
    return t


def _ld(t):
    """Leading dimension; of a single row, whose stride torch leaves open, its length."""
    return t.stride(-2) if t.shape[-2] > 1 else max(t.shape[-1], t.stride(-2))


def _int32(t, name, shape=None):
    import torch
    if t.dtype != torch.int32 or (shape is not None and (tuple(t.shape) != tuple(shape) or not t.is_contiguous())):
        raise ValueError(f"{name} must be int32{'' if shape is None else f', contiguous, of shape {tuple(shape)}'} "
                         f"(got {t.dtype}, {tuple(t.shape)}, strides {t.stride()})")
    return t


def _mx_empty(rows, k, device):
    """Codes [rows, k padded to 256, / 2] and scales [chunks, rows, 8]."""
    import torch
    chunks = (k + 255) // 256
    return (torch.empty((rows, chunks * 128), dtype=torch.uint8, device=device),
            torch.empty((chunks, rows, 8), dtype=torch.uint8, device=device))


def _mx(q, s, name, lead=()):
    """Checks codes q [*lead, rows, 128 chunks] against scales s [*lead, chunks, rows, 8]; returns (rows, k)."""
    import torch
    d = len(lead)
    if q.dtype != torch.uint8 or s.dtype != torch.uint8 or q.dim() != d + 2 or s.dim() != d + 3:
        raise ValueError(f"{name} must be uint8 codes [rows, bytes] and uint8 scales [chunks, rows, 8]"
                         + (" of every group" if d else ""))
    rows, width = q.shape[-2:]
    if tuple(q.shape[:d]) != tuple(lead) or tuple(s.shape[:d]) != tuple(lead) or width % 128 or width < 128 or rows < 1 \
            or tuple(s.shape[d:]) != (width // 128, rows, 8):
        raise ValueError(f"{name}: codes {tuple(q.shape)} do not go with scales {tuple(s.shape)}")
    if q.stride(-1) != 1 or s.stride(-1) != 1 or (rows > 1 and s.stride(-2) != 8) or \
            (s.shape[-3] > 1 and s.stride(-3) % 8):
        raise ValueError(f"{name}: codes must be row-major and scales [chunks, rows, 8] with rows contiguous")
    if d and (not s.is_contiguous() or (q.shape[0] > 1 and q.stride(0) != rows * _ld(q))):
        raise ValueError(f"{name}: the groups' codes and scales must follow one another")
    return rows, width * 2


def _lds(s):
    """Rows from one chunk's scales to the next."""
    return s.stride(-3) // 8 if s.shape[-3] > 1 else max(s.shape[-2], s.stride(-3) // 8)


def _quant_outputs(rows, cols, rowwise, colwise, device):
    if not (rowwise or colwise):
        raise ValueError("neither the row form nor the column form is asked for")
    q, s = _mx_empty(rows, cols, device) if rowwise else (None, None)
    qt, st = _mx_empty(cols, rows, device) if colwise else (None, None)
    args = []
    for c, sc, n in ((q, s, rows), (qt, st, cols)):
        args += [c.data_ptr(), c.stride(0), sc.data_ptr(), n] if c is not None else [None, 0, None, 0]
    return (q, s, qt, st), args


def quant_mxfp4_1x32(x, rowwise: bool = True, colwise: bool = False, nosat: bool = False):
    """x bf16 / fp16 / fp32 [rows, cols] -> (q, s, qt, st): MXFP4 codes uint8 [rows, 128 ceil(cols / 256)] with
    scales uint8 [ceil(cols / 256), rows, 8] of tiles along rows, and (colwise) the transposed form, codes
    [cols, 128 ceil(rows / 256)] with scales [ceil(rows / 256), cols, 8] of tiles along columns; None for a
    form not asked for. nosat: scales that never saturate an element."""
    xtype = _dtype(_matrix(x, "x"), "x")
    rows, cols = x.shape
    with _on(x):
        out, args = _quant_outputs(rows, cols, rowwise, colwise, x.device)
        fp8bq_quant_mxfp4_1x32(x.data_ptr(), xtype, rows, cols, _ld(x), *args, MX_NOSAT if nosat else 0, _stream(x))
    return out


def dispatch_mxfp4_1x32(x, src, rowwise: bool = True, colwise: bool = False, nosat: bool = False):
    """quant_mxfp4_1x32 of the rows x[src] (src int32 [rows]; an entry outside x, such as the -1 that moe_plan
    writes for padding, stands for a row of zeros)."""
    xtype = _dtype(_matrix(x, "x"), "x")
    _int32(src, "src")
    if src.dim() != 1 or src.numel() < 1 or not src.is_contiguous():
        raise ValueError("src must be a non-empty contiguous 1-D tensor")
    rows, (xrows, cols) = src.numel(), x.shape
    with _on(x, src):
        out, args = _quant_outputs(rows, cols, rowwise, colwise, x.device)
        fp8bq_dispatch_mxfp4_1x32(x.data_ptr(), xtype, xrows, cols, _ld(x), src.data_ptr(), rows, *args,
                                  MX_NOSAT if nosat else 0, _stream(x))
    return out


def dequant_mxfp4_1x32(q, s, cols, dtype=None):
    """MXFP4 codes and scales -> their values [rows, cols] in `dtype` (bfloat16 unless given)."""
    import torch
    rows, k = _mx(q, s, "q")
    dtype = torch.bfloat16 if dtype is None else dtype
    ytype = _dtype(dtype, "dtype")
    if not 1 <= cols <= k or cols <= k - 256:
        raise ValueError(f"cols must be in ({k - 256}, {k}] for codes of {q.shape[1]} bytes, got {cols}")
    with _on(q, s):
        y = torch.empty((rows, cols), dtype=dtype, device=q.device)
        fp8bq_dequant_mxfp4_1x32(q.data_ptr(), rows, cols, _ld(q), s.data_ptr(), _lds(s), y.data_ptr(), ytype, cols,
                                 _stream(q))
    return y


def _out(out, shape, dtype, device):
    """The output to write to and its type: `out` if given, else a new one."""
    import torch
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16 if dtype is None else dtype, device=device)
    elif dtype is not None and dtype != out.dtype:
        raise ValueError(f"out is {out.dtype}, dtype says {dtype}")
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"the output must be bfloat16 or float32, got {out.dtype}")
    if tuple(out.shape) != tuple(shape) or (out.shape[-1] > 1 and out.stride(-1) != 1):
        raise ValueError(f"out must be a row-major {tuple(shape)} tensor (got {tuple(out.shape)}, strides {out.stride()})")
    return out, _dtype(out, "out")


def gemm_mxfp4(a, sa, b, sb, out=None, dtype=None):
    """MXFP4 product a b^T: a codes [m, w] with scales [w / 128, m, 8], b codes [n, w] with scales [w / 128, n, 8],
    both as the quantisers write them. Returns bf16 (or `dtype`: float32) [m, n]."""
    m, k = _mx(a, sa, "a")
    n, kb = _mx(b, sb, "b")
    if k != kb:
        raise ValueError(f"a has {k} elements along the inner dimension, b {kb}")
    with _on(a, sa, b, sb, out):
        out, otype = _out(out, (m, n), dtype, a.device)
        fp8bq_gemm_mxfp4(m, n, k, a.data_ptr(), _ld(a), sa.data_ptr(), _lds(sa), b.data_ptr(), _ld(b), sb.data_ptr(),
                         _lds(sb), out.data_ptr(), otype, _ld(out), _stream(a))
    return out


def grouped_gemm_mxfp4(row_off, a, sa, b, sb, out=None, dtype=None):
    """Experts' MXFP4 products: row_off int32 [G + 1] on the GPU (moe_plan's); a [m, w]; b [G, n, w] with scales
    [G, w / 128, n, 8]. Rows row_off[e] .. row_off[e + 1] of the result [m, n] are those of a times b[e]^T;
    rows of no expert are left as they are in `out`."""
    G = b.shape[0]
    m, k = _mx(a, sa, "a")
    n, kb = _mx(b, sb, "b", (G,))
    if k != kb:
        raise ValueError(f"a has {k} elements along the inner dimension, b {kb}")
    _int32(row_off, "row_off", (G + 1,))
    with _on(a, sa, b, sb, row_off, out):
        out, otype = _out(out, (m, n), dtype, a.device)
        fp8bq_grouped_gemm_mxfp4(G, row_off.data_ptr(), m, n, k, a.data_ptr(), _ld(a), sa.data_ptr(),
                                 _lds(sa), b.data_ptr(), _ld(b), sb.data_ptr(), _lds(sb), out.data_ptr(), otype,
                                 _ld(out), _stream(a))
    return out


def grouped_wgrad_mxfp4(row_off, a, sa, b, sb, out=None, dtype=None):
    """Experts' weight gradients: a [m, w], b [n, w] the dispatched dy and x quantised along their columns (qt, st of
    dispatch_mxfp4_1x32), row_off int32 [G + 1] with multiples of 256 (moe_plan with pad=256). Returns float32
    (or `dtype`: bfloat16) [G, m, n]."""
    import torch
    m, k = _mx(a, sa, "a")
    n, kb = _mx(b, sb, "b")
    if k != kb:
        raise ValueError(f"a has {k} rows, b {kb}")
    _int32(row_off, "row_off")
    if row_off.dim() != 1 or row_off.numel() < 2 or not row_off.is_contiguous():
        raise ValueError("row_off must be contiguous, 1-D, with at least two entries")
    G = row_off.numel() - 1
    with _on(a, sa, b, sb, row_off, out):
        out, otype = _out(out, (G, m, n), torch.float32 if dtype is None and out is None else dtype, a.device)
        if G > 1 and out.stride(0) != m * _ld(out):
            raise ValueError("the experts' gradients must follow one another in out")
        fp8bq_grouped_wgrad_mxfp4(G, row_off.data_ptr(), m, n, k, a.data_ptr(), _ld(a), sa.data_ptr(),
                                  _lds(sa), b.data_ptr(), _ld(b), sb.data_ptr(), _lds(sb), out.data_ptr(), otype,
                                  _ld(out), _stream(a))
    return out


def moe_plan(idx, groups: int, pad: int = 1):
    """Dispatch plan of a router's choices idx int32 [tokens, topk] (entries outside [0, groups) are dropped) ->
    (counts int32 [groups], row_off int32 [groups + 1], src int32 [rows], pos int32 [tokens, topk]): choices per
    expert, offsets of the experts' rows (each padded to a multiple of pad), the token of each dispatched row
    (-1: none) and the row of each choice (-1: dropped); rows of an expert in the order of tokens. The number of
    rows, tokens * topk + groups * (pad - 1) rounded up to a multiple of pad, does not depend on the choices."""
    import torch
    _int32(_matrix(idx, "idx"), "idx")
    tokens, topk = idx.shape
    if groups < 1 or pad < 1:
        raise ValueError("groups and pad must be positive")
    cap = tokens * topk + groups * (pad - 1)
    cap += -cap % pad
    with _on(idx):
        new = lambda *shape: torch.empty(shape, dtype=torch.int32, device=idx.device)   # noqa: E731
        counts, row_off, src, pos = new(groups), new(groups + 1), new(cap), new(tokens, topk)
        ws = torch.empty(MOE_PLAN_WORKSPACE_BYTES, dtype=torch.uint8, device=idx.device)
        fp8bq_moe_plan(idx.data_ptr(), tokens, topk, _ld(idx), groups, pad, counts.data_ptr(), row_off.data_ptr(),
                       src.data_ptr(), cap, pos.data_ptr(), ws.data_ptr(), _stream(idx))
    return counts, row_off, src, pos


def _routing(logits, idx, score, seq_off):
    ltype = _dtype(_matrix(logits, "logits"), "logits")
    _int32(_matrix(idx, "idx"), "idx")
    if idx.shape[0] != logits.shape[0]:
        raise ValueError(f"idx has {idx.shape[0]} tokens, logits {logits.shape[0]}")
    if score not in ("softmax", "sigmoid"):
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    sequences = 1
    if seq_off is not None:
        _int32(seq_off, "seq_off")
        if seq_off.dim() != 1 or seq_off.numel() < 2 or not seq_off.is_contiguous():
            raise ValueError("seq_off must be contiguous, 1-D, with at least two entries")
        sequences = seq_off.numel() - 1
    return ltype, sequences, [logits.data_ptr(), ltype, *logits.shape, _ld(logits), idx.data_ptr(), idx.shape[1],
                              _ld(idx), seq_off.data_ptr() if seq_off is not None else None, sequences,
                              SIGMOID if score == "sigmoid" else SOFTMAX]


def moe_balance(logits, idx, coef: float, score: str = "softmax", seq_off=None):
    """Balance loss of a router: logits [tokens, experts], idx int32 [tokens, topk] the chosen experts, seq_off
    int32 [S + 1] the offsets of the sequences (None: one of all tokens) -> (loss float32 [], counts int32
    [S, experts], real int32 [S]: tokens with at least one choice)."""
    import torch
    _, sequences, args = _routing(logits, idx, score, seq_off)
    tokens, experts = logits.shape
    with _on(logits, idx, seq_off):
        loss = torch.empty((), dtype=torch.float32, device=logits.device)
        counts = torch.empty((sequences, experts), dtype=torch.int32, device=logits.device)
        real = torch.empty(sequences, dtype=torch.int32, device=logits.device)
        ws = torch.empty(fp8bq_moe_balance_workspace_size(tokens, experts, sequences), dtype=torch.uint8,
                         device=logits.device)
        fp8bq_moe_balance(*args, coef, loss.data_ptr(), counts.data_ptr(), real.data_ptr(), ws.data_ptr(),
                          _stream(logits))
    return loss, counts, real


def moe_balance_grad(dloss, logits, idx, counts, real, coef: float, score: str = "softmax", seq_off=None):
    """Gradient of moe_balance with respect to the logits, in their type; counts and real are moe_balance's, dloss
    float32 [] on the GPU."""
    import torch
    _, sequences, args = _routing(logits, idx, score, seq_off)
    _int32(counts, "counts", (sequences, logits.shape[1]))
    _int32(real, "real", (sequences,))
    if dloss.dtype != torch.float32 or dloss.numel() != 1:
        raise ValueError("dloss must be one float32 value")
    with _on(logits, idx, seq_off, counts, real, dloss):
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        fp8bq_moe_balance_grad(dloss.data_ptr(), *args, coef, counts.data_ptr(),
                               real.data_ptr(), grad.data_ptr(), logits.shape[1], _stream(logits))
    return grad
