"""The router's balance loss and its gradient over batches of many sequences, of very different lengths, empty ones
among them, with tokens before the first and behind the last, against float64."""

import numpy as np
import pytest

import fp8_fine_grained_fp8bq_amd as fb
from oracle import moe
from tests.gpu_util import log
from tests.mx_util import f64, torch_dtype

pytestmark = pytest.mark.gpu


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def offsets(kind, tokens, sequences, rng):
    if kind == "even":
        return np.arange(sequences + 1) * tokens // sequences
    if kind == "middle":                       # tokens outside at both ends
        return tokens // 3 + np.arange(sequences + 1) * (tokens // 4) // sequences
    if kind == "long first":                   # one long sequence, then short ones and empty ones
        short = np.sort(rng.integers(tokens - tokens // 8, tokens + 1, sequences))
        return np.concatenate([[0], short])
    if kind == "long last":
        short = np.sort(rng.integers(2, tokens // 8, sequences))
        return np.concatenate([short, [tokens - 1]])
    cut = np.sort(rng.integers(0, tokens + 1, sequences + 1))      # random, mostly empty where there are many
    return np.where(rng.random(len(cut)) < 0.2, cut[len(cut) // 2], cut) if sequences < 3 else cut


@pytest.mark.parametrize("kind", ["even", "middle", "long first", "long last", "random"])
@pytest.mark.parametrize("tokens,experts,topk,sequences", [(700, 60, 2, 63), (3000, 16, 3, 64), (3001, 64, 2, 65),
                                                           (9001, 8, 1, 700), (400, 70, 4, 5000), (20000, 8, 2, 4200),
                                                           (50, 256, 8, 2)])
@pytest.mark.parametrize("score,dtype", [("softmax", "float32"), ("sigmoid", "bfloat16")])
def test_many_sequences(kind, tokens, experts, topk, sequences, score, dtype):
    import torch
    log(f"balance {tokens}x{experts}, {sequences} sequences {kind} {score} {dtype}")
    rng = np.random.default_rng(tokens + sequences)
    off = np.sort(offsets(kind, tokens, sequences, rng)).astype(np.int32)
    assert len(off) == sequences + 1 and off[0] >= 0 and off[-1] <= tokens
    x = torch.from_numpy(rng.normal(0, 2, (tokens, experts))).to(torch_dtype(dtype)).cuda()
    idx = rng.integers(0, experts, (tokens, topk)).astype(np.int32)
    idx[rng.random(tokens) < 0.1] = -1
    doff, dl = dev(off), torch.tensor(1.7, device="cuda")
    loss, counts, real = fb.moe_balance(x, dev(idx), 0.3, score, doff)
    wl, wc, wr = moe.balance(f64(x), idx, 0.3, score, off)
    assert np.array_equal(counts.cpu().numpy(), wc) and np.array_equal(real.cpu().numpy(), wr)
    # every p is off by at most about 32 + experts / 64 roundings, their sums by one per addition, all terms positive
    rel = (40 + experts / 64 + tokens) * 2.0 ** -24
    assert abs(float(loss) - wl) <= rel * wl
    # The C entry writes rows of a wider table of poison: every row's own columns, none else
    buf = torch.full((tokens, experts + 5), 768.0, dtype=x.dtype, device="cuda")
    type_code = {"float32": fb.FP32, "bfloat16": fb.BF16}[dtype]
    di = dev(idx)
    fb.fp8bq_moe_balance_grad(dl.data_ptr(), x.data_ptr(), type_code, tokens, experts, experts, di.data_ptr(), topk, topk,
                              doff.data_ptr(), sequences, fb.SIGMOID if score == "sigmoid" else fb.SOFTMAX, 0.3,
                              counts.data_ptr(), real.data_ptr(), buf.data_ptr(), experts + 5,
                              torch.cuda.current_stream().cuda_stream)
    assert (buf[:, experts:] == 768.0).all()
    grad = fb.moe_balance_grad(dl, x, di, counts, real, 0.3, score, doff)
    wg = moe.balance_grad(float(dl), f64(x), idx, 0.3, score, off)
    # p (dp - sum p dp): the error is bounded by the roundings of a p and of a sum of experts positive terms, times
    # p (dp + sum p dp) <= p * 2 max dp
    p, opened = moe.scores(f64(x), score)
    top = np.zeros((tokens, 1))
    for s in range(sequences):
        if wr[s]:
            top[off[s]:off[s + 1]] = 1.7 * 0.3 / sequences * wc[s].max() * experts / (topk * wr[s] ** 2)
    tol = (64 + experts / 16) * 2.0 ** -24 * p * 2 * top
    if opened is not None:
        tol = tol * opened
    half = torch.finfo(x.dtype).eps / 2 if dtype != "float32" else 0.0
    tiny = {"bfloat16": 2.0 ** -134, "float32": 2.0 ** -149}[dtype]
    outside = np.ones(tokens, bool)
    outside[off[0]:off[-1]] = False
    for got in (f64(grad), f64(buf[:, :experts])):      # (rows of another alignment sum in another order)
        assert (np.abs(got - wg) <= tol + half * (np.abs(wg) + tol) + tiny).all()
        assert (got[outside] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("direction", ["gradient"])
def test_a_long_sequence_among_many_short_ones_takes_no_longer(direction, score):
    """The work is dealt out by tokens: 2^17 tokens take about as long in 1001 sequences of any lengths as in 8."""
    import torch
    tokens, experts = 1 << 17, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((tokens, experts), generator=gen, device="cuda")
    idx = torch.randint(0, experts, (tokens, 4), generator=gen, device="cuda", dtype=torch.int32)
    dl = torch.ones((), device="cuda")

    def times(off):
        doff = dev(np.array(off, np.int32))
        _, counts, real = fb.moe_balance(x, idx, 0.1, score, doff)
        def call():
            if direction == "forward":
                fb.moe_balance(x, idx, 0.1, score, doff)
            else:
                fb.moe_balance_grad(dl, x, idx, counts, real, 0.1, score, doff)

        best = float("inf")
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    few = times([tokens * i // 8 for i in range(9)])
    for off in ([tokens * i // 1001 for i in range(1002)], [0] + [tokens - 1000 + i for i in range(1001)],
                [tokens // 2 + i for i in range(1002)]):
        many = times(off)
        log(f"{direction} {score}: {many:.3f} ms in 1001 sequences, {few:.3f} in 8")
        # 20 times leaves room for other load; dealt out by sequences it was 50 to 500 times
        assert many <= 20 * few


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts", [8, 60, 256])
def test_gradient_of_nearly_even_loads(experts, score):
    """Counts that differ by a few in thousands: the gradient keeps its accuracy, since p (f - sum p f) does not depend
    on what f has in common; of even loads it is zero."""
    import torch
    tokens, topk = 4096 * experts // 8, 4
    rng = np.random.default_rng(experts)
    x = dev(rng.normal(size=(tokens, experts)).astype(np.float32))
    idx = (np.arange(tokens * topk) % experts).astype(np.int32).reshape(tokens, topk)
    dl = torch.ones((), device="cuda")
    _, counts, real = fb.moe_balance(x, dev(idx), 0.3, score)
    assert int(counts.min()) == int(counts.max())
    assert (fb.moe_balance_grad(dl, x, dev(idx), counts, real, 0.3, score) == 0).all()
    idx[:5, 0], idx[7, 1] = 0, 3
    _, counts, real = fb.moe_balance(x, dev(idx), 0.3, score)
    g = f64(fb.moe_balance_grad(dl, x, dev(idx), counts, real, 0.3, score))
    wg = moe.balance_grad(1.0, f64(x), idx, 0.3, score, [0, tokens])
    p, opened = moe.scores(f64(x), score)
    c = counts.cpu().numpy()[0].astype(np.float64)
    top = 0.3 * np.abs(c - c.mean()).max() * experts / (topk * tokens ** 2)
    # p (g - sum p g) with g = f - mean: every p and the sum of experts terms off by the roundings of an exponential, a
    # quotient and the additions, none of |g| above top
    tol = (64 + experts / 16) * 2.0 ** -24 * p * 2 * (top + 0.3 * experts / (topk * tokens ** 2)) * (1.0 if opened is None else opened)
    assert (np.abs(g - wg) <= tol + 2.0 ** -149).all()
