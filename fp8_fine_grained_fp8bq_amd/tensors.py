"""The MXFP4 operators, the routing of tokens to experts and the operators around a layer's Linears on torch tensors.
Reached as attributes of the package, which imports this module on their first use (the package itself does not need torch).

The calls check their arguments (ValueError), allocate the outputs and call the C entry points (Fp8bqError for their
statuses); all of that is in the extension module _tensors (csrc/torch_tensors.cpp). They run on the tensors' device,
also when it is not the current one, and on that device's current stream; every tensor of a call is on one device.
Workspaces are allocated per call, so calls on several streams and captured graphs share none.
"""

from __future__ import annotations

import torch  # noqa: F401  (its libraries have to be loaded before the extension)

from . import _tensors


def quant_mxfp4_1x32(x, rowwise: bool = True, colwise: bool = False, nosat: bool = False):
    """x bf16 / fp16 / fp32 [rows, cols] -> (q, s, qt, st): MXFP4 codes uint8 [rows, 128 ceil(cols / 256)] with
    scales uint8 [ceil(cols / 256), rows, 8] of tiles along rows, and (colwise) the transposed form, codes
    [cols, 128 ceil(rows / 256)] with scales [ceil(rows / 256), cols, 8] of tiles along columns; None for a
    form not asked for. nosat: scales that never saturate an element."""
    return _tensors.quant(x, None, rowwise, colwise, nosat)


def dispatch_mxfp4_1x32(x, src, rowwise: bool = True, colwise: bool = False, nosat: bool = False):
    """quant_mxfp4_1x32 of the rows x[src] (src int32 [rows]; an entry outside x, such as the -1 that moe_plan
    writes for padding, stands for a row of zeros; where it writes ROW_UNUSED, behind the last expert, the row form is
    left unwritten)."""
    if src is None:
        raise ValueError("src must be a tensor")
    return _tensors.quant(x, src, rowwise, colwise, nosat)


def dequant_mxfp4_1x32(q, s, cols, dtype=None):
    """MXFP4 codes and scales -> their values [rows, cols] in `dtype` (bfloat16 unless given)."""
    return _tensors.dequant(q, s, cols, dtype)


def gemm_mxfp4(a, sa, b, sb, out=None, dtype=None):
    """MXFP4 product a b^T: a codes [m, w] with scales [w / 128, m, 8], b codes [n, w] with scales [w / 128, n, 8],
    both as the quantisers write them. Returns bf16 (or `dtype`: float32) [m, n]."""
    return _tensors.gemm(a, sa, b, sb, out, dtype)


def grouped_gemm_mxfp4(row_off, a, sa, b, sb, out=None, dtype=None):
    """Experts' MXFP4 products: row_off int32 [G + 1] on the GPU (moe_plan's); a [m, w]; b [G, n, w] with scales
    [G, w / 128, n, 8]. Rows row_off[e] .. row_off[e + 1] of the result [m, n] are those of a times b[e]^T;
    rows of no expert are left as they are in `out`."""
    return _tensors.grouped_gemm(row_off, a, sa, b, sb, out, dtype)


def grouped_wgrad_mxfp4(row_off, a, sa, b, sb, out=None, dtype=None):
    """Experts' weight gradients: a [m, w], b [n, w] the dispatched dy and x quantised along their columns (qt, st of
    dispatch_mxfp4_1x32), row_off int32 [G + 1] with multiples of 256 (moe_plan with pad=256). Returns float32
    (or `dtype`: bfloat16) [G, m, n]."""
    return _tensors.grouped_wgrad(row_off, a, sa, b, sb, out, dtype)


def moe_plan(idx, groups: int, pad: int = 1):
    """Dispatch plan of a router's choices idx int32 [tokens, topk] (entries outside [0, groups) are dropped) ->
    (counts int32 [groups], row_off int32 [groups + 1], src int32 [rows], pos int32 [tokens, topk]): choices per
    expert, offsets of the experts' rows (each padded to a multiple of pad), the token of each dispatched row
    (-1: padding, ROW_UNUSED: behind the last expert) and the row of each choice (-1: dropped); rows of an expert in
    the order of tokens. The number of rows, tokens * topk + groups * (pad - 1) rounded up to a multiple of pad, does
    not depend on the choices."""
    return _tensors.moe_plan(idx, groups, pad)


def moe_balance(logits, idx, coef: float, score: str = "softmax", seq_off=None):
    """Balance loss of a router: logits [tokens, experts], idx int32 [tokens, topk] the chosen experts, seq_off
    int32 [S + 1] the offsets of the sequences (None: one of all tokens) -> (loss float32 [], counts int32
    [S, experts], real int32 [S]: tokens with at least one choice)."""
    return _tensors.moe_balance(logits, idx, coef, score, seq_off)


def moe_balance_grad(dloss, logits, idx, counts, real, coef: float, score: str = "softmax", seq_off=None):
    """Gradient of moe_balance with respect to the logits, in their type; counts and real are moe_balance's, dloss
    float32 [] on the GPU."""
    return _tensors.moe_balance_grad(dloss, logits, idx, counts, real, coef, score, seq_off)


def rmsnorm(x, weight, eps: float = 1e-6, residual=None, quant: bool = True, norm: bool = False, pow2: bool = False):
    """RMS norm of the rows of x (bf16 / fp16 / fp32 [rows, cols]) after adding `residual` -> (q, s, y, h, rstd): codes
    uint8 [rows, cols] and scales float32 [cols / 128, rows] for the next FP8 Linear (quant; pow2: power-of-two scales),
    the normalised rows in x's type (norm), x + residual in x's type, and float32 [rows]; None for what is not asked
    for. weight [cols] of any of the three types."""
    return _tensors.rmsnorm(x, weight, eps, residual, quant, norm, pow2)


def rmsnorm_grad(dy, h, weight, rstd, dh=None):
    """Gradient of rmsnorm: dy of the normalised rows, h (x itself where there was no residual) and rstd as rmsnorm
    returned them, dh what reaches h besides -> (dx in h's type, the gradient of x and of the residual; dweight float32
    [cols])."""
    return _tensors.rmsnorm_grad(dy, h, weight, rstd, dh)


def moe_dispatch(x, src, pos, s=None, out=None, s_out=None):
    """Tokens to the rows of a plan (src and pos are moe_plan's): x bf16 / fp16 / fp32 [tokens, cols], or uint8 codes with
    their scales s float32 [cols / 128, tokens] -> (rows [len(src), cols], their scales [cols / 128, len(src)] or None).
    Padding rows are zeros, rows behind the last expert are left as they are in `out` and `s_out`. Its gradient is
    moe_combine(drows, pos)."""
    return _tensors.moe_dispatch(x, src, pos, s, out, s_out)


def moe_combine(y, pos, weight=None, base=None, out=None):
    """Rows y [rows, cols] back to their tokens: base[t] + the sum of weight[t, j] * y[pos[t, j]] over the choices that
    have a row, in y's type [tokens, cols]. weight float32 [tokens, topk] (None: ones); base in y's type (None: zeros).
    y may have no rows, as where every choice is another GPU's."""
    return _tensors.moe_combine(y, pos, weight, base, out)


def moe_combine_grad(dout, y, pos, weight, src, out=None):
    """Gradient of moe_combine -> (dy [rows, cols] in y's type, dweight float32 [tokens, topk]); padding rows of dy are
    zeros, rows behind the last expert are left as they are in `out`. base's gradient is dout."""
    return _tensors.moe_combine_grad(dout, y, pos, weight, src, out)


def gemv_mxfp4(x, w, ws, out=None, dtype=None):
    """Product of a few rows x (bf16 / fp16 / fp32 [m, k], kept as they are) with an MXFP4 weight: codes w [n, 128 ceil(k /
    256)] with scales ws -> [m, n] in x's type (or `dtype`)."""
    return _tensors.gemv(x, w, ws, out, dtype)


def grouped_gemv_mxfp4(row_off, x, w, ws, src=None, out=None, dtype=None):
    """The same over experts: rows row_off[e] .. row_off[e + 1] of the result are those of x[src] (x without src) times
    expert e's weight w[e]^T; row_off int32 [G + 1] and src int32 [rows] on the GPU (moe_plan's). Rows of no expert are
    left as they are in `out`."""
    return _tensors.grouped_gemv(row_off, x, w, ws, src, out, dtype)
