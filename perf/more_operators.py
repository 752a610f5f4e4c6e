"""What stands around the block-scaled Linears of a layer, as cases to measure.

Operators: the RMS norm with the residual's addition whose output is the FP8 Linear's operand (E4M3 codes and scales of
1x128 tiles), and its gradient; tokens brought to their experts' rows and back with the gates' weights, and the gradient;
the product of a few unquantised rows with a resident 4-bit (MXFP4) weight, dense and over experts.

Layouts (those of the package): FP8 scales are float32 [cols / 128, rows]; MXFP4 codes are two to a byte, the element with
the even index in the low four bits, in rows padded with zero codes to a multiple of 256 elements, their scales E8M0 bytes
[chunk of 256 elements][row][8]; a dispatch plan has the offsets of the experts' rows, the token of each row (-1: padding,
-2: behind the last expert) and the row of each choice (-1: none).
"""

import math

import torch

own = False

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one generated token on its way into an FP8 Linear
        {"name": "norm-token", "op": "norm", "rows": 1, "cols": 7168, "residual": True, "quant": True, "norm": False,
         "type": "bf16"},
        # a long batch: codes for the FP8 Linear and the 16-bit rows that the router reads
        {"name": "norm-prompt", "op": "norm", "rows": 16384, "cols": 7168, "residual": True, "quant": True, "norm": True,
         "type": "bf16"},
        # odd sizes: a plain norm, half precision, rows that start at any address
        {"name": "norm-ragged", "op": "norm", "rows": 1003, "cols": 1057, "residual": False, "quant": False, "norm": True,
         "type": "fp16"},
        # a training step's norm, there and back
        {"name": "norm-step", "op": "norm_step", "rows": 4096, "cols": 7168, "residual": True, "quant": True, "norm": False,
         "type": "bf16"},
        # the same of a short fp32 batch
        {"name": "norm-step-short", "op": "norm_step", "rows": 333, "cols": 2048, "residual": True, "quant": True,
         "norm": False, "type": "fp32"},
        # generated tokens to 32 of 256 experts and back: FP8 codes out, 16-bit results in, added to the residual
        {"name": "route-decode", "op": "route", "tokens": 256, "topk": 8, "experts": 256, "local": 32, "cols": 7168,
         "zipf": 1.1, "pad": 128},
        # a prompt, every expert here
        {"name": "route-prompt", "op": "route", "tokens": 8192, "topk": 8, "experts": 64, "local": 64, "cols": 7168,
         "zipf": 0.5, "pad": 128},
        # a training step: rows out and back, gradients of rows, gates and tokens
        {"name": "route-step", "op": "route_step", "tokens": 4096, "topk": 4, "experts": 32, "local": 32, "cols": 2048,
         "zipf": 0.5, "pad": 256, "type": "bf16"},
        # odd sizes, fp32, a quarter of the experts here
        {"name": "route-step-odd", "op": "route_step", "tokens": 333, "topk": 6, "experts": 160, "local": 40, "cols": 1057,
         "zipf": 1.1, "pad": 1, "type": "fp32"},
        # one token against a resident 4-bit weight
        {"name": "product-token", "op": "product", "m": 1, "n": 2048, "k": 7168, "type": "bf16"},
        # a small serving batch against a wide one
        {"name": "product-batch", "op": "product", "m": 12, "n": 18432, "k": 7168, "type": "fp16"},
        # generated tokens through 32 of 256 experts
        {"name": "experts-token", "op": "experts", "tokens": 32, "topk": 8, "experts": 256, "local": 32, "n": 2048,
         "k": 7168, "zipf": 1.1, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_step", "route", "route_step", "product", "product", "experts"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_step"):
        quant = rng.random() < 0.6
        cols = 128 * _log(rng, 1, 64) if quant else _log(rng, 33, 8192)
        return {"op": op, "rows": _log(rng, 1, min(16384, (16384 if op == "norm" else 4096) * 7168 // cols) // (2 if kind == "fp32" else 1)),
                "cols": cols, "residual": rng.random() < 0.6, "quant": quant, "norm": not quant or rng.random() < 0.4, "type": kind}
    if op in ("route", "route_step"):
        local = rng.choice([4, 8, 16, 32, 40, 64])
        case = {"op": op, "tokens": _log(rng, 1, 8192 if op == "route" else 4096), "topk": rng.randint(1, 8),
                "experts": local * rng.choice([1, 2, 4]), "local": local, "zipf": rng.choice([0.0, 0.5, 1.1]),
                "pad": rng.choice([1, 128, 256])}
        if op == "route":
            return {**case, "cols": 128 * _log(rng, 1, 56)}
        return {**case, "cols": _log(rng, 33, 1024), "type": kind}
    if op == "product":
        return {"op": op, "m": _log(rng, 1, 48), "n": _log(rng, 64, 16384), "k": _log(rng, 32, 7168), "type": kind}
    local = rng.choice([4, 8, 16, 32])
    return {"op": op, "tokens": _log(rng, 1, 48), "topk": rng.randint(1, 8), "experts": local * rng.choice([1, 2, 8]), "local": local,
            "n": _log(rng, 64, 2048), "k": _log(rng, 64, 7168), "zipf": rng.choice([0.0, 0.5, 1.1]), "type": kind}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _normal(gen, shape, std, dtype, outliers=0.0):
    x = torch.randn(shape, generator=gen, device="cuda")
    if outliers:
        x = torch.where(torch.rand(shape, generator=gen, device="cuda") < outliers, x * 50, x)
    return (x * std).to(dtype)


def _choices(gen, tokens, topk, experts, zipf):
    """Distinct experts of each token, drawn with probabilities (i + 1)^-zipf."""
    logp = -zipf * torch.log(torch.arange(1, experts + 1, device="cuda", dtype=torch.float32))
    u = torch.rand((tokens, experts), generator=gen, device="cuda").clamp_(1e-20, 1.0 - 1e-7)
    return torch.topk(logp - torch.log(-torch.log(u)), min(topk, experts), dim=1).indices


def _plan(idx, groups, pad):
    """Offsets (each group padded to `pad` rows), token of each row and row of each choice; rows of a group in the order
    of tokens."""
    flat = idx.flatten()
    key = torch.where(flat < groups, flat, groups)
    counts = torch.bincount(key, minlength=groups + 1)[:groups]
    off = torch.nn.functional.pad(((counts + pad - 1) // pad * pad).cumsum(0), (1, 0))
    order = torch.argsort(key, stable=True)
    first = torch.nn.functional.pad(counts.cumsum(0), (1, 0))
    sorted_key = key[order]
    row = off[sorted_key] + torch.arange(flat.numel(), device=idx.device) - first[sorted_key]
    row = torch.where(sorted_key < groups, row, -1)
    pos = torch.empty_like(flat)
    pos[order] = row
    cap = flat.numel() + groups * (pad - 1)
    cap += -cap % pad
    src = torch.where(torch.arange(cap + 1, device=idx.device) < off[-1], -1, -2)
    src[row] = order // idx.shape[1]                  # row -1: the spare last entry
    return off.to(torch.int32), src[:-1].to(torch.int32), pos.reshape(idx.shape).to(torch.int32)


def _weight(gen, shape):
    """A weight [..., n, k] in MXFP4: codes [..., n, k padded to 256, / 2] and scales [..., k padded / 256, n, 8]."""
    k = shape[-1]
    w = _normal(gen, shape, 0.02, torch.bfloat16)
    t = torch.nn.functional.pad(w, (0, -k % 256)).unflatten(-1, (-1, 32)).float()
    e = torch.where(t.abs().amax(-1) == 0, -127, torch.frexp(t.abs().amax(-1))[1] - 3)
    a = torch.ldexp(t, -e.unsqueeze(-1)).abs()
    a = (torch.round(a / torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))) * torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))).clamp(max=6)
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = torch.where(torch.signbit(t), code | 8, code).flatten(-2)
    s = (e + 127).to(torch.uint8).unflatten(-1, (-1, 8)).transpose(-2, -3)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), s.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    op, kind = case["op"], _TYPES[case.get("type", "bf16")]
    if op in ("norm", "norm_step"):
        shape = (case["rows"], case["cols"])
        st["x"] = _normal(gen, shape, 0.5, kind, 1e-3)
        st["residual"] = _normal(gen, shape, 2.0, kind) if case["residual"] else None
        st["weight"] = (1 + 0.2 * torch.randn(case["cols"], generator=gen, device="cuda")).to(kind)
        if op == "norm_step":
            st["dy"] = _normal(gen, shape, 1e-3, kind)
            st["dh"] = _normal(gen, shape, 1e-3, kind) if case["residual"] else None    # what comes down the residual stream
    elif op in ("route", "route_step"):
        t, k, c = case["tokens"], min(case["topk"], case["experts"]), case["cols"]
        idx = _choices(gen, t, k, case["experts"], case["zipf"])
        _, st["src"], st["pos"] = _plan(idx, case["local"], case["pad"])
        st["gate"] = torch.softmax(torch.randn((t, k), generator=gen, device="cuda"), 1)
        rows = st["src"].numel()
        st["y"] = _normal(gen, (rows, c), 1.0, kind)
        st["base"] = _normal(gen, (t, c), 1.0, kind)
        if op == "route":
            # a batch as an FP8 quantiser leaves it: codes of magnitudes up to 448, a scale for each tile
            st["q"] = (torch.randn((t, c), generator=gen, device="cuda") * 140).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            st["s"] = torch.rand((c // 128, t), generator=gen, device="cuda") * 1e-2 + 1e-3
            st["q_rows"] = torch.zeros((rows, c), dtype=torch.uint8, device="cuda")
            st["s_rows"] = torch.zeros((c // 128, rows), device="cuda")
        else:
            st["x"] = _normal(gen, (t, c), 1.0, kind)
            st["x_rows"] = torch.zeros((rows, c), dtype=kind, device="cuda")
            st["dout"] = _normal(gen, (t, c), 1e-3, kind)
            st["dx_rows"] = _normal(gen, (rows, c), 1e-3, kind)
            st["dy_rows"] = torch.zeros((rows, c), dtype=kind, device="cuda")
    elif op == "product":
        st["x"] = _normal(gen, (case["m"], case["k"]), 1.0, kind, 1e-3)
        st["w"], st["ws"] = _weight(gen, (case["n"], case["k"]))
    else:
        idx = _choices(gen, case["tokens"], case["topk"], case["experts"], case["zipf"])
        st["off"], st["src"], _ = _plan(idx, case["local"], 1)
        st["x"] = _normal(gen, (case["tokens"], case["k"]), 1.0, kind, 1e-3)
        st["w"], st["ws"] = _weight(gen, (case["local"], case["n"], case["k"]))
        st["y"] = torch.zeros((st["src"].numel(), case["n"]), dtype=kind, device="cuda")
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _norm(st):
    x = st["x"].float()
    if st["residual"] is not None:
        x = x + st["residual"].float()
    rstd = torch.rsqrt((x * x).mean(1) + _EPS)
    y = x * rstd[:, None] * st["weight"].float()
    out = [rstd]
    if st["residual"] is not None:
        out.append(x.to(st["x"].dtype))
    if st["case"]["norm"]:
        out.append(y.to(st["x"].dtype))
    if st["case"]["quant"]:
        t = y.unflatten(1, (-1, 128))
        s = t.abs().amax(2) / 448
        q = torch.where(s[:, :, None] == 0, t, t / s[:, :, None])
        out += [q.to(torch.float8_e4m3fn).flatten(1), s.t().contiguous()]
    return out


def _decode(q, s, k):
    """Float32 values of MXFP4 codes and scales, [..., rows, k]."""
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), device=q.device)
    v = torch.stack((grid[(q & 15).int()], grid[(q >> 4).int()]), -1).flatten(-2)
    e = s.transpose(-2, -3).flatten(-2).to(torch.int32) - 127
    return torch.ldexp(v, e.repeat_interleave(32, -1))[..., :k]


def _to_rows(x, src):
    """Row r is x[src[r]], of zeros where there is none."""
    return torch.where((src >= 0)[:, None], x[src.clamp(min=0).long()], torch.zeros((), dtype=x.dtype, device=x.device))


def _back(y, pos, gate, base):
    """Sum over a token's choices of their rows, weighted, and what the token has besides."""
    rows = torch.where((pos >= 0)[:, :, None], y[pos.clamp(min=0).long()].float(), 0.0)
    if gate is not None:
        rows = rows * gate[:, :, None]
    out = rows.sum(1)
    return out if base is None else out + base.float()


def _run_plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "norm":
        return _norm(st)
    if op == "norm_step":
        out = _norm(st)
        rstd = out[0][:, None]
        h = (out[1] if case["residual"] else st["x"]).float()
        dy = st["dy"].float()
        hat = h * rstd
        g = dy * st["weight"].float()
        dx = rstd * (g - hat * (g * hat).mean(1, keepdim=True))
        if st["dh"] is not None:
            dx = dx + st["dh"].float()
        return out + [dx.to(st["x"].dtype), (dy * hat).sum(0)]
    if op == "route":
        rows = _to_rows(st["q"], st["src"]).view(torch.float8_e4m3fn)
        s = _to_rows(st["s"].t(), st["src"]).t().contiguous()
        return rows, s, _back(st["y"], st["pos"], st["gate"], st["base"]).to(st["y"].dtype)
    if op == "route_step":
        kind, pos, src = st["y"].dtype, st["pos"], st["src"]
        rows = _to_rows(st["x"], src)
        out = _back(st["y"], pos, st["gate"], st["base"]).to(kind)
        d = st["dout"].float()
        mine = pos >= 0
        dgate = torch.where(mine, (st["y"][pos.clamp(min=0).long()].float() * d[:, None]).sum(2), 0.0)
        gate_of_row = torch.zeros(len(src) + 1, device=src.device)
        gate_of_row[torch.where(mine, pos, len(src)).long()] = st["gate"]
        dy = _to_rows(d, src) * gate_of_row[:-1, None]
        return rows, out, dy.to(kind), dgate, _back(st["dx_rows"], pos, None, None).to(kind)
    if op == "product":
        return (st["x"].float() @ _decode(st["w"], st["ws"], case["k"]).t()).to(st["x"].dtype)
    # every expert's rows in a block of their own, as many as there are tokens at most
    off, x = st["off"].long(), st["x"].float()
    place = torch.arange(case["tokens"], device=x.device) + off[:-1, None]
    inside = place < off[1:, None]
    token = st["src"].long()[place.clamp(max=len(st["src"]) - 1)].clamp(min=0)
    y = torch.matmul(x[token], _decode(st["w"], st["ws"], case["k"]).transpose(1, 2).contiguous())
    out = torch.zeros((len(st["src"]) + 1, case["n"]), device=x.device)
    out[torch.where(inside, place, len(st["src"])).flatten()] = y.flatten(0, 1)
    return out[:-1].to(st["x"].dtype)


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------

def _own_norm(fb, st):
    case = st["case"]
    q, s, y, h, rstd = fb.rmsnorm(st["x"], st["weight"], _EPS, residual=st["residual"], quant=case["quant"], norm=case["norm"])
    out = [v for v in (rstd, h, y) if v is not None]
    if case["quant"]:
        out += [q.view(torch.float8_e4m3fn), s]
    return out


def _run_own(st):
    import fp8_fine_grained_fp8bq_amd as fb
    case, op = st["case"], st["case"]["op"]
    if op == "norm":
        return _own_norm(fb, st)
    if op == "norm_step":
        out = _own_norm(fb, st)
        h = out[1] if case["residual"] else st["x"]
        return out + list(fb.rmsnorm_grad(st["dy"], h, st["weight"], out[0], dh=st["dh"]))
    if op == "route":
        rows, s = fb.moe_dispatch(st["q"], st["src"], st["pos"], s=st["s"], out=st["q_rows"], s_out=st["s_rows"])
        return rows.view(torch.float8_e4m3fn), s, fb.moe_combine(st["y"], st["pos"], st["gate"], base=st["base"])
    if op == "route_step":
        rows, _ = fb.moe_dispatch(st["x"], st["src"], st["pos"], out=st["x_rows"])
        out = fb.moe_combine(st["y"], st["pos"], st["gate"], base=st["base"])
        dy, dgate = fb.moe_combine_grad(st["dout"], st["y"], st["pos"], st["gate"], st["src"], out=st["dy_rows"])
        return rows, out, dy, dgate, fb.moe_combine(st["dx_rows"], st["pos"])
    if op == "product":
        return fb.gemv_mxfp4(st["x"], st["w"], st["ws"])
    return fb.grouped_gemv_mxfp4(st["off"], st["x"], st["w"], st["ws"], src=st["src"], out=st["y"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _e4m3(v):
    """The nearest value of 1 + 4 + 3 bits (bias 7), ties to the even mantissa."""
    a = v.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    n = torch.floor(a / step)
    left = a / step - n
    n = n + torch.where(left == 0.5, n % 2, (left > 0.5).to(n.dtype))
    return torch.copysign(n * step, v)


def _exact_codes(q, s, k):
    low, high = (q % 16).long(), (q // 16).long()
    code = torch.empty((*q.shape[:-1], 2 * q.shape[-1]), dtype=torch.int64, device=q.device)
    code[..., 0::2], code[..., 1::2] = low, high
    grid = torch.tensor(_GRID, dtype=torch.float64, device=q.device)
    v = grid[code % 8] * (1 - 2 * (code // 8))
    b = s.movedim(-3, -2).reshape(*v.shape[:-1], -1, 1).double()
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(b - 127)).flatten(-2)[..., :k]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_step"):
        x = st["x"].double()
        h = x
        if case["residual"]:
            x = x + st["residual"].double()
            h = x.to(st["x"].dtype).double()           # held in the rows' type
        rstd = 1 / torch.sqrt((x ** 2).sum(1) / case["cols"] + _EPS)
        y = torch.einsum("rc,r,c->rc", x, rstd, st["weight"].double())
        out = [rstd]
        if case["residual"]:
            out.append(x)
        if case["norm"]:
            out.append(y)
        if case["quant"]:
            s = y.abs().unflatten(1, (-1, 128)).max(2).values / 448
            out += [_e4m3(y / s.clamp(min=1e-300).repeat_interleave(128, 1)), s.t().contiguous()]
        if op == "norm_step":
            g = st["dy"].double() * st["weight"].double()
            # d/dx of x / sqrt(mean x^2 + eps), the mean's part through the dot product with the row
            dot = (g * h).sum(1) / case["cols"]
            dx = g * rstd[:, None] - h * (dot * rstd ** 3)[:, None]
            if st["dh"] is not None:
                dx = dx + st["dh"].double()
            out += [dx, torch.einsum("rc,rc,r->c", st["dy"].double(), h, rstd)]
        return out
    if op in ("route", "route_step"):
        pos, src = st["pos"].long(), st["src"].long()
        t, j = (pos >= 0).nonzero(as_tuple=True)
        at = pos[t, j]
        out = st["base"].double()
        out.index_put_((t,), st["y"][at].double() * st["gate"][t, j].double()[:, None], accumulate=True)
        if op == "route":
            rows = torch.zeros((len(src), case["cols"]), dtype=torch.float64, device="cuda")
            s = torch.zeros((case["cols"] // 128, len(src)), dtype=torch.float64, device="cuda")
            rows[at] = st["q"].view(torch.float8_e4m3fn).double()[t]
            s[:, at] = st["s"].double()[:, t]
            return rows, s, out
        rows = torch.zeros((len(src), case["cols"]), dtype=torch.float64, device="cuda")
        rows[at] = st["x"][t].double()
        dy = torch.zeros_like(rows)
        dy[at] = st["dout"][t].double() * st["gate"][t, j].double()[:, None]
        dgate = torch.zeros(pos.shape, dtype=torch.float64, device="cuda")
        dgate[t, j] = torch.einsum("rc,rc->r", st["dout"][t].double(), st["y"][at].double())
        dx = torch.zeros((case["tokens"], case["cols"]), dtype=torch.float64, device="cuda")
        dx.index_add_(0, t, st["dx_rows"][at].double())
        return rows, out, dy, dgate, dx
    w = _exact_codes(st["w"], st["ws"], case["k"])
    if op == "product":
        return st["x"].double() @ w.t()
    off, token = st["off"].tolist(), st["src"].tolist()
    y = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["local"]):
        y[off[e]:off[e + 1]] = st["x"][token[off[e]:off[e + 1]]].double() @ w[e].t()
    return y


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

_MX = 17 / 32     # bytes of a 4-bit element: half a byte of code, a scale byte for 32


def _share(case):
    """How many of the tokens' choices the experts here are expected to get, and how many of these experts get any."""
    p = [(i + 1) ** -case["zipf"] for i in range(case["experts"])]
    k = min(case["topk"], case["experts"])
    total = sum(p)
    lo, hi = 0.0, 1e4
    for _ in range(60):       # expert i is among k distinct draws with about 1 - (1 - p)^c, c so that these sum to k
        c = (lo + hi) / 2
        lo, hi = (c, hi) if sum(1 - (1 - v / total) ** c for v in p) < k else (lo, c)
    mine = [1 - (1 - v / total) ** lo for v in p[: case["local"]]]
    return case["tokens"] * sum(mine), sum(1 - (1 - v) ** case["tokens"] for v in mine)


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case.get("type", "bf16")]
    op = case["op"]
    if op in ("norm", "norm_step"):
        n = case["rows"] * case["cols"]
        parts = 1 + 2 * case["residual"] + case["norm"]
        move = n * (size * parts + (1 + 4 / 128) * case["quant"])
        if op == "norm_step":
            # dy, dh and dx; h is still the forward pass's, x where there is no residual
            move += n * size * (2 + case["residual"] + 1) + 4 * case["cols"]
            return {"bytes": move, "flops": 18 * n}
        return {"bytes": move, "flops": 6 * n}
    if op in ("route", "route_step"):
        t, c = case["tokens"], case["cols"]
        rows = _share(case)[0]
        ints = 8 * t * case["topk"]
        if op == "route":
            return {"bytes": ints + (t + rows) * c * (1 + 4 / 128) + (rows + 2 * t) * c * 2, "flops": 2 * rows * c}
        # dispatch x; combine y with base; dout, y again and dy; the dispatched rows' gradients
        return {"bytes": ints + c * size * ((t + rows) + (rows + 2 * t) + (t + 2 * rows) + (rows + t)), "flops": 6 * rows * c}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * k * _MX + m * (n + k) * size, "flops": 2 * m * n * k}
    rows, used = _share(case)
    n, k = case["n"], case["k"]
    return {"bytes": used * n * k * _MX + (min(case["tokens"], rows) * k + rows * n) * size, "flops": 2 * rows * n * k}
