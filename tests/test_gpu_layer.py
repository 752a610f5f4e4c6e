"""The operators around a layer's Linears together, as a layer runs them: a step with experts forward and back, generated
tokens, the same captured in graphs and on two streams at once."""

import numpy as np
import pytest

import fp8_fine_grained_fp8bq_amd as fb
from oracle import e4m3, layer, moe, mxfp4
from tests.gpu_util import log
from tests.layer_util import ROW, U, check, f64, matrix, rounded

pytestmark = pytest.mark.gpu


def weights_fp8(seed, experts, n, k):
    """Per-expert FP8 weights as the package quantises them, and their values."""
    import torch
    rng = np.random.default_rng(seed)
    q, s = [], []
    for _ in range(experts):
        w = torch.from_numpy(rng.normal(0, 0.05, (n, k))).bfloat16().cuda()
        a, b, _ = fb.quant_w_128x128(w)
        q.append(a)
        s.append(b)
    q, s = torch.stack(q), torch.stack(s)
    values = e4m3.decode(q.cpu().numpy()) * np.kron(f64(s), np.ones((128, 128)))
    return q, s, values


def router(seed, tokens, experts, topk):
    """Choices and gates of random logits."""
    import torch
    rng = np.random.default_rng(seed)
    top = torch.from_numpy(rng.normal(size=(tokens, experts))).float().cuda().topk(topk, 1)
    return top.indices.to(torch.int32), torch.softmax(top.values, 1)


def rows_of(q, s):
    """Values of E4M3 codes with 1x128 scales."""
    return e4m3.decode(q.cpu().numpy()) * np.repeat(f64(s).T, 128, 1)


def test_layer_of_experts():
    """norm -> plan -> dispatch of the codes -> the experts' FP8 product -> combine onto the residual, each step against
    the float64 form of what it was given."""
    tokens, cols, experts, topk = 200, 512, 6, 2
    x, r = matrix(1, tokens, cols), matrix(2, tokens, cols, std=2.0)
    w = matrix(3, 1, cols, "float32", 0.2)[0].contiguous() + 1
    wq, ws, vw = weights_fp8(4, experts, cols, cols)
    idx, gate = router(5, tokens, experts, topk)
    q, s, y, h, rstd = fb.rmsnorm(x, w, residual=r, norm=True)
    counts, off, src, pos = fb.moe_plan(idx, experts, pad=128)
    qd, sd = fb.moe_dispatch(q, src, pos, s=s)
    rows = int(off[-1])
    out = fb.grouped_gemm(off.tolist(), qd[:rows], sd[:, :rows].contiguous(), wq, ws)
    got = f64(fb.moe_combine(out, pos, gate, base=h))

    n_off, n_src, n_pos = (t.cpu().numpy() for t in (off, src, pos))
    wh, _, wy = layer.rmsnorm(f64(x), f64(r), f64(w), 1e-6)
    vq = rows_of(q, s)
    assert (np.abs(vq - wy) <= 2.0 ** -4 * np.abs(wy) * 1.01 + 2.0 ** -10 * np.repeat(f64(s).T, 128, 1)).all()   # half a step of E4M3
    given = layer.dispatch(vq, n_pos, n_src, len(n_src), 0.0)[:rows]
    assert np.array_equal(rows_of(qd[:rows], sd[:, :rows]), given)
    want = np.concatenate([given[n_off[e]:n_off[e + 1]] @ vw[e].T for e in range(experts)])
    mag = np.concatenate([np.abs(given[n_off[e]:n_off[e + 1]]) @ np.abs(vw[e]).T for e in range(experts)])
    check("product", f64(out), want, rounded(want, 2e-3 * mag, "bfloat16"))
    total, terms = layer.combine(f64(out), n_pos, f64(gate), f64(h))
    check("layer", got, total, rounded(total, (topk + 1) * U * terms, "bfloat16"))


def test_training_step_gradients():
    """The whole chain in fp32 against the float64 gradient of the same chain written as matrices: norm, dispatch, one
    fixed matrix per expert, combine onto the residual."""
    import torch
    tokens, cols, experts, topk = 60, 192, 5, 3
    x, r, dout = (matrix(s, tokens, cols, "float32") for s in (11, 12, 13))
    w = matrix(14, 1, cols, "float32", 0.2)[0].contiguous() + 1
    idx, gate = router(15, tokens, experts, topk)
    _, off, src, pos = fb.moe_plan(idx, experts, pad=32)
    m = np.random.default_rng(16).normal(0, cols ** -0.5, (experts, cols, cols))
    n_off, n_pos = off.cpu().numpy(), pos.cpu().numpy()

    def experts_of(rows, back):
        """The experts' matrices in float64, rounded to fp32 once (what stands for their products here)."""
        v = rows.double()
        out = torch.zeros_like(v)
        for e in range(experts):
            a = torch.from_numpy(m[e]).cuda()
            out[n_off[e]:n_off[e + 1]] = v[n_off[e]:n_off[e + 1]] @ (a if back else a.t())
        return out.float()

    _, _, y, h, rstd = fb.rmsnorm(x, w, residual=r, quant=False, norm=True)
    rows, _ = fb.moe_dispatch(y, src, pos)
    z = experts_of(rows, False)
    out = fb.moe_combine(z, pos, gate, base=h)
    dz, dgate = fb.moe_combine_grad(dout, z, pos, gate, src)
    dy = fb.moe_combine(experts_of(dz, True), pos)
    dx, dw = fb.rmsnorm_grad(dy, h, w, rstd, dh=dout)

    leaves = [t.double().detach().requires_grad_() for t in (x, w, gate)]
    lx, lw, lg = leaves
    hh = lx + r.double()
    yy = hh * (hh.square().mean(1, keepdim=True) + 1e-6).rsqrt() * lw
    per = torch.stack([yy @ torch.from_numpy(m[e]).cuda().t() for e in range(experts)])
    total = hh + (lg[:, :, None] * per[idx.long(), torch.arange(tokens, device="cuda")[:, None]]).sum(1)
    total.backward(dout.double())
    # each of the chain's roundings is at most (topk + ROW / U + 64) U of the norm of what it goes through; the chain has six
    # steps, and what amplifies them (rstd, gates and matrices of norm about 1 to 3) is far below the 100 allowed for it
    rel = 6 * (topk + ROW / U + 64) * U * 100
    for name, a, b in (("out", out, total.detach()), ("dx", dx, lx.grad), ("dw", dw, lw.grad), ("dgate", dgate, lg.grad)):
        err = (a.double() - b).norm() / b.norm()
        assert err <= rel, (name, float(err), rel)
    assert np.array_equal(n_pos >= 0, np.ones_like(n_pos, bool))


def generate(x, r, w, idx, gate, wq, ws, experts):
    """Generated tokens through a layer with 4-bit experts."""
    _, _, y, h, _ = fb.rmsnorm(x, w, residual=r, quant=False, norm=True)
    _, off, src, pos = fb.moe_plan(idx, experts)
    z = fb.grouped_gemv_mxfp4(off, y, wq, ws, src=src)
    return fb.moe_combine(z, pos, gate, base=h)


def generated(seed, tokens, cols, experts, topk, dtype="bfloat16"):
    import torch
    x, r = matrix(seed, tokens, cols, dtype), matrix(seed + 1, tokens, cols, dtype)
    w = matrix(seed + 2, 1, cols, dtype, 0.2)[0].contiguous() + 1
    idx, gate = router(seed + 3, tokens, experts, topk)
    rng = np.random.default_rng(seed + 4)
    packed = [mxfp4.quantise(rng.normal(0, 0.05, (cols, cols))) for _ in range(experts)]
    wq, ws = (torch.from_numpy(np.stack([p[i] for p in packed])).cuda() for i in (0, 1))
    return x, r, w, idx, gate, wq, ws, experts


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_generated_tokens(tokens):
    cols, experts, topk = 384, 8, 2
    args = generated(20 + tokens, tokens, cols, experts, topk, "float32")
    got = f64(generate(*args))
    x, r, w, idx, gate, wq, ws, _ = args
    h, _, y = layer.rmsnorm(f64(x), f64(r), f64(w), 1e-6)
    values = [mxfp4.values(wq[e].cpu().numpy(), ws[e].cpu().numpy(), cols) for e in range(experts)]
    want, mag = h.copy(), np.abs(h)
    for t in range(tokens):
        for j in range(topk):
            e, g = int(idx[t, j]), float(gate[t, j])
            want[t] += g * (values[e] @ y[t])
            mag[t] += g * (np.abs(values[e]) @ np.abs(y[t]))
    check("tokens", got, want, (3 * cols + 64) * 2.0 ** -23 * mag + 2 * ROW * mag)


def test_captured_in_a_graph():
    """Captured once, replayed with new inputs and eager work between: every replay equals the eager result."""
    import torch
    args = generated(40, 24, 512, 16, 4)
    x = args[0]
    h, dy, w = matrix(50, 300, 640), matrix(51, 300, 640), matrix(52, 1, 640, "float32")[0].contiguous()

    def step():
        out = generate(*args)
        q, s, _, _, rstd = fb.rmsnorm(h, w)
        dx, dw = fb.rmsnorm_grad(dy, h, w, rstd)
        _, _, src, pos = fb.moe_plan(args[3], 16, pad=8)
        rows, _ = fb.moe_dispatch(x, src, pos)
        dz, dg = fb.moe_combine_grad(x, rows, pos, args[4], src)
        return [out, q, s, dx, dw, dg, fb.moe_combine(rows, pos), fb.moe_combine(dz, pos)]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    log("graph capture of the layer's operators")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for i in range(4):
        x.copy_(matrix(60 + i, *x.shape))
        h.copy_(matrix(70 + i, *h.shape))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b), f"replay {i}"


def test_two_streams_at_once():
    """Calls on two streams share nothing."""
    import torch
    sets = [generated(80 + 10 * i, 30 + i, 512, 8, 2) for i in range(2)]
    grads = [(matrix(100 + i, 700, 1024), matrix(110 + i, 700, 1024), matrix(120 + i, 1, 1024, "float32")[0].contiguous()) for i in range(2)]

    def work(i):
        h, dy, w = grads[i]
        out = [generate(*sets[i])]
        rstd = fb.rmsnorm(h, w)[4]
        return out + list(fb.rmsnorm_grad(dy, h, w, rstd))

    want = [work(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(work(i))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))


def test_balance_of_the_same_plan():
    """The router's choices that the plan takes also feed the balance loss: the counts agree."""
    import torch
    rng = np.random.default_rng(7)
    logits = torch.from_numpy(rng.normal(size=(90, 12))).float().cuda()
    idx = logits.topk(3, 1).indices.to(torch.int32)
    counts, off, src, pos = fb.moe_plan(idx, 12, pad=4)
    _, c, real = fb.moe_balance(logits, idx, 0.1)
    assert torch.equal(c[0], counts) and int(real) == 90
    ones = torch.ones((90, 8), device="cuda")
    rows, _ = fb.moe_dispatch(ones, src, pos)
    used = moe.plan(idx.cpu().numpy(), 12, 4, src.numel())[2]
    assert np.array_equal((f64(rows)[used != -2] == 1).all(1), used[used != -2] >= 0)


@pytest.mark.parametrize("tokens,topk", [(1, 1), (40, 3)])
def test_layer_without_rows(tokens, topk):
    """Every choice is another GPU's: the experts have no rows, and the layer returns its residual stream."""
    import torch
    cols, experts = 384, 5
    log(f"layer of {tokens} tokens without rows")
    x, r, dout = matrix(130, tokens, cols), matrix(131, tokens, cols), matrix(132, tokens, cols)
    w = matrix(133, 1, cols, "float32", 0.2)[0].contiguous() + 1
    wq, ws, _ = weights_fp8(134, experts, cols, cols)
    idx = torch.full((tokens, topk), -1, dtype=torch.int32, device="cuda")
    gate = torch.ones((tokens, topk), device="cuda")
    q, s, y, h, rstd = fb.rmsnorm(x, w, residual=r, norm=True)
    counts, off, src, pos = fb.moe_plan(idx, experts, pad=128)
    rows = int(off[-1])
    assert rows == 0 and (counts == 0).all()
    qd, sd = fb.moe_dispatch(q, src, pos, s=s)
    for product in (fb.grouped_gemm, fb.grouped_gemm_decode):
        z = product(off.tolist(), qd[:rows], sd[:, :rows].contiguous(), wq, ws)
        assert z.shape == (0, cols)
    z = fb.grouped_gemm_decode(off.tolist(), qd[:rows], sd[:, :rows].contiguous(), wq, ws, split=False)
    assert torch.equal(fb.moe_combine(z, pos, gate, base=h), h)
    assert (fb.moe_combine(z, pos, gate) == 0).all()
    dz, dgate = fb.moe_combine_grad(dout, z, pos, gate, src[:rows])
    assert dz.shape == (0, cols) and dgate.shape == (tokens, topk) and (dgate == 0).all()
    dy = fb.moe_combine(dz, pos, base=y)
    assert torch.equal(dy, y)
    dx, dw = fb.rmsnorm_grad(dy, h, w, rstd, dh=dout)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    out = torch.full((tokens, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(fb.moe_combine(z, pos, out=out), torch.zeros_like(out))


def test_training_step_within_its_roundings():
    """The same chain, element by element: each step's roundings (those of its own test) carried through the steps behind it
    to first order, 1% for the higher ones."""
    import torch
    tokens, cols, experts, topk = 60, 192, 5, 3
    x, r, dout = (matrix(s, tokens, cols, "float32") for s in (211, 212, 213))
    w = matrix(214, 1, cols, "float32", 0.2)[0].contiguous() + 1
    idx, gate = router(215, tokens, experts, topk)
    _, off, src, pos = fb.moe_plan(idx, experts, pad=32)
    m = np.random.default_rng(216).normal(0, cols ** -0.5, (experts, cols, cols))
    n_off, n_src, n_pos = (t.cpu().numpy() for t in (off, src, pos))
    rows = len(n_src)

    def experts_of(v, back=False, mat=m):
        out = np.zeros_like(v)
        for e in range(experts):
            out[n_off[e]:n_off[e + 1]] = v[n_off[e]:n_off[e + 1]] @ (mat[e] if back else mat[e].T)
        return out

    def product(t, back=False):
        return torch.from_numpy(experts_of(f64(t), back)).float().cuda()

    _, _, y, h, rstd = fb.rmsnorm(x, w, residual=r, quant=False, norm=True)
    z = product(fb.moe_dispatch(y, src, pos)[0])
    out = fb.moe_combine(z, pos, gate, base=h)
    dz, dgate = fb.moe_combine_grad(dout, z, pos, gate, src)
    dz[off[-1]:] = 0                                                   # behind the last expert, not written
    dy = fb.moe_combine(product(dz, True), pos)
    dx, dw = fb.rmsnorm_grad(dy, h, w, rstd, dh=dout)

    # the chain in float64, and beside every value what the fp32 one may be off by
    RSTD = ROW / 2 + 4 * U
    size = np.abs(m)
    vw, vg, vd = f64(w), f64(gate), f64(dout)
    wh, wr, wy = layer.rmsnorm(f64(x), f64(r), vw, 1e-6)
    ey = (RSTD + 4 * U) * np.abs(wy)
    to_rows = lambda v: layer.dispatch(v, n_pos, n_src, rows, 0.0)  # noqa: E731
    wz = experts_of(to_rows(wy))
    ez = experts_of(to_rows(ey), mat=size) + U * np.abs(wz)
    wout, mag = layer.combine(wz, n_pos, vg, wh)
    check("out", f64(out), wout, 1.01 * (layer.combine(ez, n_pos, vg, None)[0] + (topk + 1) * U * mag + 2 * U * np.abs(wh)))
    wdz, wdg, mag = layer.combine_grad(vd, wz, n_pos, vg)
    check("dgate", f64(dgate), wdg, 1.01 * (layer.combine_grad(np.abs(vd), ez, n_pos, vg)[1] + ROW * mag))
    wrows = experts_of(wdz, True)
    erows = experts_of(U * np.abs(wdz), True, size) + U * np.abs(wrows)
    wdy, mag = layer.combine(wrows, n_pos, None, None)
    edy = layer.combine(erows, n_pos, None, None)[0] + topk * U * mag
    check("dy", f64(dy), wdy, 1.01 * edy)
    wdx, wdw = layer.rmsnorm_grad(wdy, wh, vw, wr, vd)
    hat, g, eg = np.abs(wh) * wr[:, None], np.abs(wdy * vw), edy * np.abs(vw)
    whole = wr[:, None] * (g + hat * (g * hat).mean(1, keepdims=True))          # of dx's terms; each has rstd up to three times
    edx = wr[:, None] * (eg + hat * (eg * hat).mean(1, keepdims=True)) + (3 * RSTD + 2 * U + ROW + 8 * U) * whole + 2 * U * np.abs(wdx)
    check("dx", f64(dx), wdx, 1.01 * edx)
    check("dw", f64(dw), wdw, 1.01 * ((edy * hat).sum(0) + (RSTD + U + (tokens + 600) * U) * np.abs(wdy * hat).sum(0)))
