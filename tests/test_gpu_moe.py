"""Routing on the GPU: the dispatch plan entry by entry, the balance loss and its gradient against float64, and the
whole chain of a router with its experts."""

import numpy as np
import pytest

import fp8_fine_grained_fp8bq_amd as fb
from oracle import moe, mxfp4
from tests.gpu_util import log
from tests.mx_util import check_product, codes, f64, matrix, torch_dtype

pytestmark = pytest.mark.gpu


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("pad", [1, 32, 256])
@pytest.mark.parametrize("tokens,topk,groups", [(1, 1, 1), (1, 8, 256), (7, 3, 5), (64, 2, 8), (257, 8, 32), (700, 3, 100),
                                                (1000, 8, 256), (5000, 5, 17)])
def test_plan(tokens, topk, groups, pad):
    log(f"plan {tokens}x{topk} groups {groups} pad {pad}")
    rng = np.random.default_rng(tokens + groups)
    idx = (rng.zipf(1.3, (tokens, topk)) % (groups + groups // 3 + 2) - 1).astype(np.int32)
    idx[rng.random(idx.shape) < 0.05] = 1 << 30
    counts, off, src, pos = fb.moe_plan(dev(idx), groups, pad)
    wc, wo, ws, wp = moe.plan(idx, groups, pad, src.numel())
    assert np.array_equal(counts.cpu().numpy(), wc) and np.array_equal(off.cpu().numpy(), wo)
    assert np.array_equal(pos.cpu().numpy(), wp) and np.array_equal(src.cpu().numpy(), ws)


@pytest.mark.parametrize("value", [-1, 0, 3, 9])
def test_plan_of_equal_choices(value):
    """Every choice the same expert, or none inside."""
    idx = np.full((3000, 2), value, np.int32)
    got = fb.moe_plan(dev(idx), 4, 32)
    for g, w in zip(got, moe.plan(idx, 4, 32, got[2].numel())):
        assert np.array_equal(g.cpu().numpy(), w)


def test_plan_of_strided_choices_and_many():
    rng = np.random.default_rng(1)
    wide = rng.integers(-2, 70, (70000, 10)).astype(np.int32)
    got = fb.moe_plan(dev(wide)[:, 2:10], 64, 1)
    idx = wide[:, 2:10]
    ok = (idx >= 0) & (idx < 64)
    flat = np.where(ok, idx, 64).flatten()
    order = np.argsort(flat, kind="stable")[:ok.sum()]
    assert np.array_equal(got[0].cpu().numpy(), np.bincount(flat, minlength=65)[:64])
    src = got[2].cpu().numpy()
    assert np.array_equal(src[:len(order)], order // 8) and (src[len(order):] == fb.ROW_UNUSED).all()
    pos = got[3].cpu().numpy().flatten()
    assert np.array_equal(pos[order], np.arange(len(order))) and (pos[~ok.flatten()] == -1).all()


CASES = [(1, 1, 1, [0, 1]), (5, 2, 1, [0, 5]), (64, 60, 6, [0, 64]), (333, 64, 6, [0, 100, 100, 290]),
         (200, 256, 8, [10, 11, 60, 190]), (300, 160, 3, [0, 300]), (128, 400, 4, [0, 64, 128]), (90, 1000, 8, [5, 80]),
         (700, 8, 2, list(range(0, 701, 7))), (50, 100, 70, [0, 50]), (9, 130, 128, [0, 3, 3, 9])]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,topk,off", CASES, ids=lambda v: str(v)[:16])
def test_balance(tokens, experts, topk, off, score, dtype):
    import torch
    log(f"balance {tokens}x{experts} {score} {dtype}")
    rng = np.random.default_rng(tokens + experts)
    x = torch.from_numpy(rng.normal(0, 2, (tokens, experts))).to(torch_dtype(dtype)).cuda()
    idx = rng.integers(0, experts, (tokens, topk)).astype(np.int32)
    idx[rng.random(idx.shape) < 0.1] = -1
    idx[rng.random(tokens) < 0.1] = experts + 5            # tokens without a choice
    loss, counts, real = fb.moe_balance(x, dev(idx), 0.3, score, dev(np.array(off, np.int32)))
    wl, wc, wr = moe.balance(f64(x), idx, 0.3, score, off)
    assert np.array_equal(counts.cpu().numpy(), wc) and np.array_equal(real.cpu().numpy(), wr)
    # every p is off by at most about 32 + experts / 64 roundings (exponential, sums over lanes, quotient), their sums over
    # tokens by one per addition (at most tokens), all terms positive
    rel = (40 + experts / 64 + tokens) * 2.0 ** -24
    assert abs(float(loss) - wl) <= rel * wl
    dl = torch.tensor(1.7, device="cuda")
    grad = fb.moe_balance_grad(dl, x, dev(idx), counts, real, 0.3, score, dev(np.array(off, np.int32)))
    assert grad.dtype == x.dtype
    wg = moe.balance_grad(float(dl), f64(x), idx, 0.3, score, off)
    # p (dp - sum p dp): each factor off by the roundings of a p and of a sum of experts positive terms, so the error is
    # bounded by p (dp + sum p dp) <= p * 2 max dp
    p, opened = moe.scores(f64(x), score)
    top = np.zeros((tokens, 1))
    for s in range(len(off) - 1):
        if wr[s]:
            top[off[s]:off[s + 1]] = 1.7 * 0.3 / (len(off) - 1) * wc[s].max() * experts / (topk * wr[s] ** 2)
    tol = (64 + experts / 16) * 2.0 ** -24 * p * 2 * top
    if opened is not None:
        tol = tol * opened
    half = torch.finfo(x.dtype).eps / 2 if dtype != "float32" else 0.0
    tiny = {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -134, "float32": 2.0 ** -149}[dtype]
    assert (np.abs(f64(grad) - wg) <= tol + half * (np.abs(wg) + tol) + tiny).all()
    again = fb.moe_balance_grad(dl, x, dev(idx), counts, real, 0.3, score, dev(np.array(off, np.int32)))
    assert (grad == again).all() and fb.moe_balance(x, dev(idx), 0.3, score, dev(np.array(off, np.int32)))[0] == loss


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_masked_experts_and_strides(score):
    """-inf logits (masked experts, a whole token of them), NaN in tokens that take no part, rows of a wider table."""
    import torch
    rng = np.random.default_rng(4)
    wide = rng.normal(size=(60, 41)).astype(np.float32)
    x = wide[:, 3:39]
    x[:, 5] = -np.inf
    x[10] = -np.inf
    x[20:22] = 50.0
    idx = rng.integers(0, 36, (60, 4)).astype(np.int32)
    idx[30] = -1
    x[30] = np.nan
    x[55:] = np.nan
    off = [0, 33, 55]
    dx = dev(wide)[:, 3:39]
    loss, counts, real = fb.moe_balance(dx, dev(idx), 0.3, score, dev(np.array(off, np.int32)))
    clean = np.where(np.isnan(x), 0, x).astype(np.float64)
    wl, wc, wr = moe.balance(clean, idx, 0.3, score, off)
    assert np.array_equal(counts.cpu().numpy(), wc) and abs(float(loss) - wl) <= 200 * 2.0 ** -24 * wl
    g = f64(fb.moe_balance_grad(torch.ones((), device="cuda"), dx, dev(idx), counts, real, 0.3, score,
                                dev(np.array(off, np.int32))))
    wg = moe.balance_grad(1.0, clean, idx, 0.3, score, off)
    assert np.isfinite(g).all() and (g[30] == 0).all() and (g[55:] == 0).all() and (g[10] == 0).all()
    assert np.abs(g - wg).max() <= 100 * 2.0 ** -24 * np.abs(wg).max() * 10


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts", [5, 64, 200])
def test_balance_shows_a_nan(score, experts):
    """A token whose logits are NaN, one of them or all, makes the loss and its own gradients NaN and no others'."""
    import torch
    rng = np.random.default_rng(experts)
    clean = rng.normal(size=(70, experts)).astype(np.float32)
    idx = dev(rng.integers(0, experts, (70, 2)).astype(np.int32))
    one = torch.ones((), device="cuda")
    _, counts, real = fb.moe_balance(dev(clean), idx, 1.0, score)
    want = fb.moe_balance_grad(one, dev(clean), idx, counts, real, 1.0, score)
    for where in (slice(None), slice(experts - 1, experts)):
        x = clean.copy()
        x[33, where] = np.nan
        loss, c, r = fb.moe_balance(dev(x), idx, 1.0, score)
        assert torch.isnan(loss) and (c == counts).all() and (r == real).all()
        g = fb.moe_balance_grad(one, dev(x), idx, counts, real, 1.0, score)
        assert torch.isnan(g[33]).all()
        keep = torch.arange(70, device="cuda") != 33
        assert (g[keep] == want[keep]).all()


def test_balance_gradient_against_differences():
    import torch
    rng = np.random.default_rng(6)
    x = dev(rng.normal(size=(40, 12)).astype(np.float32))
    idx = dev(rng.integers(0, 12, (40, 3)).astype(np.int32))
    for score in ("softmax", "sigmoid"):
        _, counts, real = fb.moe_balance(x, idx, 1.0, score)
        g = f64(fb.moe_balance_grad(torch.ones((), device="cuda"), x, idx, counts, real, 1.0, score))
        d = rng.normal(size=(40, 12))
        h = 0.05
        up = float(fb.moe_balance(x + dev(d.astype(np.float32)) * h, idx, 1.0, score)[0])
        dn = float(fb.moe_balance(x - dev(d.astype(np.float32)) * h, idx, 1.0, score)[0])
        # the loss is about 1: the difference quotient carries 2^-24 / h of rounding and O(h^2) of curvature
        assert abs((up - dn) / (2 * h) - (g * d).sum()) <= 2 * 2.0 ** -24 / h + 0.02 * h


@pytest.mark.parametrize("tokens,topk,experts,n,k", [(1, 2, 4, 64, 96), (50, 2, 4, 160, 288), (300, 4, 16, 96, 256)])
def test_chain_of_a_router_with_its_experts(tokens, topk, experts, n, k):
    """Plan, dispatch, experts' products, their gradients and the balance loss together, eager and replayed as a graph
    with other choices."""
    import torch

    def inputs(seed):
        rng = np.random.default_rng(seed)
        logits = dev(rng.normal(size=(tokens, experts)).astype(np.float32))
        return (matrix(seed, tokens, k), matrix(seed + 50, tokens, n, std=1e-2), logits,
                torch.topk(logits, topk, 1).indices.int())

    w = [matrix(90 + e, n, k, std=0.1) for e in range(experts)]
    forms = [fb.quant_mxfp4_1x32(v, colwise=True) for v in w]
    wq, ws, wqt, wst = (torch.stack([f[i] for f in forms]) for i in range(4))
    dl = torch.ones((), device="cuda")

    def step(x, dy, logits, idx):
        counts, off, src, pos = fb.moe_plan(idx, experts, pad=256)
        xq, xs, xqt, xst = fb.dispatch_mxfp4_1x32(x, src, colwise=True)
        gq, gs, gqt, gst = fb.dispatch_mxfp4_1x32(dy, src, colwise=True)
        y = fb.grouped_gemm_mxfp4(off, xq, xs, wq, ws)
        dx = fb.grouped_gemm_mxfp4(off, gq, gs, wqt, wst)
        dw = fb.grouped_wgrad_mxfp4(off, gqt, gst, xqt, xst)
        loss, cnt, real = fb.moe_balance(logits, idx, 0.01)
        dlogits = fb.moe_balance_grad(dl, logits, idx, cnt, real, 0.01)
        rows = pos.long()
        return counts, off, pos, y[rows], dx[rows], dw, loss, dlogits, cnt

    def check(x, dy, logits, idx, got):
        counts, off, pos, y, dx, dw, loss, dlogits, cnt = got
        hidx = idx.cpu().numpy()
        assert np.array_equal(counts.cpu().numpy(), np.bincount(hidx.flatten(), minlength=experts))
        assert np.array_equal(cnt.cpu().numpy()[0], counts.cpu().numpy())
        vx = mxfp4.values(*mxfp4.quantise(f64(x)), k)
        vg = mxfp4.values(*mxfp4.quantise(f64(dy)), n)
        for e in range(experts):
            t, j = np.nonzero(hidx == e)
            if len(t):
                check_product(f64(y)[t, j], vx[t], codes(wq[e], ws[e], k), k, "bfloat16")
                check_product(f64(dx)[t, j], vg[t], codes(wqt[e], wst[e], n), n, "bfloat16")
            pad = -(-max(len(t), 1) // 256) * 256
            xt, gt = np.zeros((k, pad)), np.zeros((n, pad))
            xt[:, :len(t)], gt[:, :len(t)] = f64(x)[t].T, f64(dy)[t].T
            check_product(f64(dw[e]), mxfp4.values(*mxfp4.quantise(gt), pad), mxfp4.values(*mxfp4.quantise(xt), pad), pad,
                          "float32")
        want = moe.balance(f64(logits), hidx, 0.01, "softmax", [0, tokens])[0]
        assert abs(float(loss) - want) <= (100 + tokens) * 2.0 ** -24 * want

    first = inputs(1)
    check(*first, step(*first))
    bufs = [t.clone() for t in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*bufs)
    for seed in (2, 3, 4):
        new = inputs(seed)
        for b, v in zip(bufs, new):
            b.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        check(*new, out)
        eager = step(*new)
        assert all((a == b).all() for a, b in zip(out, eager))


def test_calls_on_two_streams_at_once():
    """Plans, dispatches (each row read once) and balance losses of two batches, side by side on two streams, many
    times over: each stream's results are those of the batch alone."""
    import torch
    tokens, topk, experts, k = 2048, 4, 16, 2048

    def batch(seed):
        rng = np.random.default_rng(seed)
        logits = dev(rng.normal(size=(tokens, experts)).astype(np.float32))
        return matrix(seed, tokens, k), logits, torch.topk(logits, topk, 1).indices.int()

    def work(x, logits, idx):
        _, off, src, pos = fb.moe_plan(idx, experts)
        q, s, _, _ = fb.dispatch_mxfp4_1x32(x, src)
        rows = pos.flatten().long()
        loss, counts, _ = fb.moe_balance(logits, idx, 0.1)
        return off, src, pos, q[rows], s[:, rows], loss, counts

    batches = [batch(1), batch(2)]
    want = [work(*b) for b in batches]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for b, st in zip(batches, streams):
            with torch.cuda.stream(st):
                got.append(work(*b))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all((a == b).all() for a, b in zip(g, w))
