"""The MXFP4 operators and the routing of tokens to experts on torch tensors: checks of what the C entry points cannot
see, allocation of the outputs, and the call. Reached as attributes of the package, which imports this module on their
first use (the package itself does not need torch).

The calls run on the tensors' device (also when it is not the current one) and on that device's current stream; every
tensor of a call is on one device. Workspaces are allocated per call, so calls on several streams and captured graphs
share none.
"""

from __future__ import annotations

import torch

from . import (BF16, FP16, FP32, MOE_PLAN_WORKSPACE_BYTES, MX_NOSAT, SIGMOID, SOFTMAX, fp8bq_dequant_mxfp4_1x32,
               fp8bq_dispatch_mxfp4_1x32, fp8bq_gemm_mxfp4, fp8bq_grouped_gemm_mxfp4, fp8bq_grouped_wgrad_mxfp4,
               fp8bq_moe_balance, fp8bq_moe_balance_grad, fp8bq_moe_balance_workspace_size, fp8bq_moe_plan,
               fp8bq_quant_mxfp4_1x32)


def _raw_stream(t):
    """The current stream of t's device as an int (the stream object that _stream makes costs a microsecond)."""
    return torch._C._cuda_getCurrentRawStream(t.device.index)


class _Current:
    """Stands in for a device guard where the device is current already (a guard costs microseconds)."""

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        return False


_CURRENT = _Current()


def _on(*tensors):
    """The one device of the tensors, made current for the call."""
    dev = tensors[0].device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {t.device}")
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on the GPU, got {dev}")
    return _CURRENT if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


_DTYPES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}


def _dtype(t, name):
    dtype = getattr(t, "dtype", t)
    if dtype not in _DTYPES:
        raise ValueError(f"{name} must be bfloat16, float16 or float32 (got {dtype})")
    return _DTYPES[dtype]


def _matrix(t, name):
    shape = t.shape
    if len(shape) != 2 or not shape[0] or not shape[1] or (t.stride(1) != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be a non-empty 2-D row-major tensor (got {tuple(shape)}, strides {t.stride()})")
    return t


def _ld(t):
    """Leading dimension; of a single row, whose stride torch leaves open, its length."""
    shape = t.shape
    return shape[-1] if t.is_contiguous() else t.stride(-2) if shape[-2] > 1 else max(shape[-1], t.stride(-2))


def _int32(t, name, shape=None):
    if t.dtype != torch.int32 or (shape is not None and (tuple(t.shape) != tuple(shape) or not t.is_contiguous())):
        raise ValueError(f"{name} must be int32{'' if shape is None else f', contiguous, of shape {tuple(shape)}'} "
                         f"(got {t.dtype}, {tuple(t.shape)}, strides {t.stride()})")
    return t


def _mx_empty(rows, k, like):
    """Codes [rows, k padded to 256, / 2] and scales [chunks, rows, 8]."""
    chunks = (k + 255) // 256
    return (like.new_empty((rows, chunks * 128), dtype=torch.uint8),
            like.new_empty((chunks, rows, 8), dtype=torch.uint8))


def _mx(q, s, name, lead=()):
    """Checks codes q [*lead, rows, 128 chunks] against scales s [*lead, chunks, rows, 8]; returns (rows, k)."""
    qs, ss, d = q.shape, s.shape, len(lead)
    if q.dtype != torch.uint8 or s.dtype != torch.uint8 or len(qs) != d + 2 or len(ss) != d + 3:
        raise ValueError(f"{name} must be uint8 codes [rows, bytes] and uint8 scales [chunks, rows, 8]"
                         + (" of every group" if d else ""))
    rows, width = qs[-2:]
    chunks = width >> 7
    if not rows or not chunks or width & 127 or qs[:d] != lead or ss != (*lead, chunks, rows, 8):
        raise ValueError(f"{name}: codes {tuple(qs)} do not go with scales {tuple(ss)}")
    if q.is_contiguous() and s.is_contiguous():
        return rows, width * 2
    if q.stride(-1) != 1 or s.stride(-1) != 1 or (rows > 1 and s.stride(-2) != 8) or \
            (chunks > 1 and s.stride(-3) % 8):
        raise ValueError(f"{name}: codes must be row-major and scales [chunks, rows, 8] with rows contiguous")
    if d and (not s.is_contiguous() or (qs[0] > 1 and q.stride(0) != rows * _ld(q))):
        raise ValueError(f"{name}: the groups' codes and scales must follow one another")
    return rows, width * 2


def _lds(s):
    """Rows from one chunk's scales to the next."""
    shape = s.shape
    return shape[-2] if s.is_contiguous() else s.stride(-3) // 8 if shape[-3] > 1 else max(shape[-2], s.stride(-3) // 8)


def _quant_outputs(rows, cols, rowwise, colwise, like):
    if not (rowwise or colwise):
        raise ValueError("neither the row form nor the column form is asked for")
    q = s = qt = st = None
    args = [None, 0, None, 0, None, 0, None, 0]
    if rowwise:
        q, s = _mx_empty(rows, cols, like)
        args[:4] = q.data_ptr(), q.shape[1], s.data_ptr(), rows
    if colwise:
        qt, st = _mx_empty(cols, rows, like)
        args[4:] = qt.data_ptr(), qt.shape[1], st.data_ptr(), cols
    return (q, s, qt, st), args


def quant_mxfp4_1x32(x, rowwise: bool = True, colwise: bool = False, nosat: bool = False):
    """x bf16 / fp16 / fp32 [rows, cols] -> (q, s, qt, st): MXFP4 codes uint8 [rows, 128 ceil(cols / 256)] with
    scales uint8 [ceil(cols / 256), rows, 8] of tiles along rows, and (colwise) the transposed form, codes
    [cols, 128 ceil(rows / 256)] with scales [ceil(rows / 256), cols, 8] of tiles along columns; None for a
    form not asked for. nosat: scales that never saturate an element."""
    xtype = _dtype(_matrix(x, "x"), "x")
    rows, cols = x.shape
    with _on(x):
        out, args = _quant_outputs(rows, cols, rowwise, colwise, x)
        fp8bq_quant_mxfp4_1x32(x.data_ptr(), xtype, rows, cols, _ld(x), *args, MX_NOSAT if nosat else 0, _raw_stream(x))
    return out


def dispatch_mxfp4_1x32(x, src, rowwise: bool = True, colwise: bool = False, nosat: bool = False):
    """quant_mxfp4_1x32 of the rows x[src] (src int32 [rows]; an entry outside x, such as the -1 that moe_plan
    writes for padding, stands for a row of zeros; where it writes ROW_UNUSED, behind the last expert, the row form is
    left unwritten)."""
    xtype = _dtype(_matrix(x, "x"), "x")
    _int32(src, "src")
    if src.dim() != 1 or src.numel() < 1 or not src.is_contiguous():
        raise ValueError("src must be a non-empty contiguous 1-D tensor")
    rows, (xrows, cols) = src.numel(), x.shape
    with _on(x, src):
        out, args = _quant_outputs(rows, cols, rowwise, colwise, x)
        # rows that several experts get are read once where that is worth two more launches: 16384 tokens of 7168, 131072
        # choices of which 54066 are here: 86 us against 203
        ws = src.new_empty(xrows + rows) if not colwise and rows >= 2 * xrows and xrows * cols >= 1 << 22 else None
        fp8bq_dispatch_mxfp4_1x32(x.data_ptr(), xtype, xrows, cols, _ld(x), src.data_ptr(), rows, *args,
                                  MX_NOSAT if nosat else 0, None if ws is None else ws.data_ptr(), _raw_stream(x))
    return out


def dequant_mxfp4_1x32(q, s, cols, dtype=None):
    """MXFP4 codes and scales -> their values [rows, cols] in `dtype` (bfloat16 unless given)."""
    rows, k = _mx(q, s, "q")
    dtype = torch.bfloat16 if dtype is None else dtype
    ytype = _dtype(dtype, "dtype")
    if not 1 <= cols <= k or cols <= k - 256:
        raise ValueError(f"cols must be in ({k - 256}, {k}] for codes of {q.shape[1]} bytes, got {cols}")
    with _on(q, s):
        y = q.new_empty((rows, cols), dtype=dtype)
        fp8bq_dequant_mxfp4_1x32(q.data_ptr(), rows, cols, _ld(q), s.data_ptr(), _lds(s), y.data_ptr(), ytype, cols,
                                 _raw_stream(q))
    return y


def _out(out, shape, dtype, like):
    """The output to write to and its type: `out` if given, else a new one."""
    if out is None:
        dtype = torch.bfloat16 if dtype is None else dtype
        otype = _dtype(dtype, "dtype")
        if otype == FP16:
            raise ValueError(f"the output must be bfloat16 or float32, got {dtype}")
        return like.new_empty(shape, dtype=dtype), otype
    if dtype is not None and dtype != out.dtype:
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
        out, otype = _out(out, (m, n), dtype, a)
        fp8bq_gemm_mxfp4(m, n, k, a.data_ptr(), _ld(a), sa.data_ptr(), _lds(sa), b.data_ptr(), _ld(b), sb.data_ptr(),
                         _lds(sb), out.data_ptr(), otype, _ld(out), _raw_stream(a))
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
        out, otype = _out(out, (m, n), dtype, a)
        fp8bq_grouped_gemm_mxfp4(G, row_off.data_ptr(), m, n, k, a.data_ptr(), _ld(a), sa.data_ptr(),
                                 _lds(sa), b.data_ptr(), _ld(b), sb.data_ptr(), _lds(sb), out.data_ptr(), otype,
                                 _ld(out), _raw_stream(a))
    return out


def grouped_wgrad_mxfp4(row_off, a, sa, b, sb, out=None, dtype=None):
    """Experts' weight gradients: a [m, w], b [n, w] the dispatched dy and x quantised along their columns (qt, st of
    dispatch_mxfp4_1x32), row_off int32 [G + 1] with multiples of 256 (moe_plan with pad=256). Returns float32
    (or `dtype`: bfloat16) [G, m, n]."""
    m, k = _mx(a, sa, "a")
    n, kb = _mx(b, sb, "b")
    if k != kb:
        raise ValueError(f"a has {k} rows, b {kb}")
    _int32(row_off, "row_off")
    if row_off.dim() != 1 or row_off.numel() < 2 or not row_off.is_contiguous():
        raise ValueError("row_off must be contiguous, 1-D, with at least two entries")
    G = row_off.numel() - 1
    with _on(a, sa, b, sb, row_off, out):
        out, otype = _out(out, (G, m, n), torch.float32 if dtype is None and out is None else dtype, a)
        if G > 1 and out.stride(0) != m * _ld(out):
            raise ValueError("the experts' gradients must follow one another in out")
        fp8bq_grouped_wgrad_mxfp4(G, row_off.data_ptr(), m, n, k, a.data_ptr(), _ld(a), sa.data_ptr(),
                                  _lds(sa), b.data_ptr(), _ld(b), sb.data_ptr(), _lds(sb), out.data_ptr(), otype,
                                  _ld(out), _raw_stream(a))
    return out


def moe_plan(idx, groups: int, pad: int = 1):
    """Dispatch plan of a router's choices idx int32 [tokens, topk] (entries outside [0, groups) are dropped) ->
    (counts int32 [groups], row_off int32 [groups + 1], src int32 [rows], pos int32 [tokens, topk]): choices per
    expert, offsets of the experts' rows (each padded to a multiple of pad), the token of each dispatched row
    (-1: padding, ROW_UNUSED: behind the last expert) and the row of each choice (-1: dropped); rows of an expert in the order of tokens. The number of
    rows, tokens * topk + groups * (pad - 1) rounded up to a multiple of pad, does not depend on the choices."""
    _int32(_matrix(idx, "idx"), "idx")
    tokens, topk = idx.shape
    if groups < 1 or pad < 1:
        raise ValueError("groups and pad must be positive")
    cap = tokens * topk + groups * (pad - 1)
    cap += -cap % pad
    with _on(idx):
        counts, row_off, src, pos = (idx.new_empty(n) for n in (groups, groups + 1, cap, (tokens, topk)))
        ws = idx.new_empty(MOE_PLAN_WORKSPACE_BYTES // 4)
        fp8bq_moe_plan(idx.data_ptr(), tokens, topk, _ld(idx), groups, pad, counts.data_ptr(), row_off.data_ptr(),
                       src.data_ptr(), cap, pos.data_ptr(), ws.data_ptr(), _raw_stream(idx))
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
    _, sequences, args = _routing(logits, idx, score, seq_off)
    tokens, experts = logits.shape
    with _on(logits, idx, seq_off):
        loss = logits.new_empty((), dtype=torch.float32)
        counts, real = idx.new_empty((sequences, experts)), idx.new_empty(sequences)
        ws = idx.new_empty(fp8bq_moe_balance_workspace_size(tokens, experts, sequences) // 4)
        fp8bq_moe_balance(*args, coef, loss.data_ptr(), counts.data_ptr(), real.data_ptr(), ws.data_ptr(),
                          _raw_stream(logits))
    return loss, counts, real


def moe_balance_grad(dloss, logits, idx, counts, real, coef: float, score: str = "softmax", seq_off=None):
    """Gradient of moe_balance with respect to the logits, in their type; counts and real are moe_balance's, dloss
    float32 [] on the GPU."""
    _, sequences, args = _routing(logits, idx, score, seq_off)
    _int32(counts, "counts", (sequences, logits.shape[1]))
    _int32(real, "real", (sequences,))
    if dloss.dtype != torch.float32 or dloss.numel() != 1:
        raise ValueError("dloss must be one float32 value")
    with _on(logits, idx, seq_off, counts, real, dloss):
        grad = logits.new_empty(logits.shape)
        fp8bq_moe_balance_grad(dloss.data_ptr(), *args, coef, counts.data_ptr(),
                               real.data_ptr(), grad.data_ptr(), logits.shape[1], _raw_stream(logits))
    return grad
