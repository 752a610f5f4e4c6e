"""Dispatch of a batch large enough for the tensor layer to read each row once, and of one just below, against the form
that gathers every row: the same bytes in every row of an expert, alone, on two streams at once, and replayed."""

import pytest

import fp8_fine_grained_fp8bq_amd as fb
from tests.gpu_util import log

pytestmark = pytest.mark.gpu


def gathered(x, src):
    """The row form through the C entry without a workspace."""
    import torch
    rows, (xrows, cols) = src.numel(), x.shape
    chunks = -(-cols // 256)
    q = torch.empty((rows, chunks * 128), dtype=torch.uint8, device="cuda")
    s = torch.empty((chunks, rows, 8), dtype=torch.uint8, device="cuda")
    fb.fp8bq_dispatch_mxfp4_1x32(x.data_ptr(), fb.BF16, xrows, cols, x.stride(0), src.data_ptr(), rows, q.data_ptr(), q.shape[1],
                                 s.data_ptr(), rows, None, 0, None, 0, 0, None, torch.cuda.current_stream().cuda_stream)
    return q, s


def batch(seed, tokens, cols, experts, skew):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((tokens, cols), generator=gen, device="cuda").bfloat16()
    idx = torch.randint(0, experts, (tokens, 8), generator=gen, device="cuda", dtype=torch.int32)
    if skew:
        idx[: tokens // 4] = 1                         # a token's eight choices the same expert, and more
    _, off, src, _ = fb.moe_plan(idx, min(experts, 8), pad=3)
    return x, off, src


@pytest.mark.parametrize("tokens,cols", [(4096, 3001), (4096, 3110), (12290, 1025), (1755, 7168), (1756, 7168)])
@pytest.mark.parametrize("experts,skew", [(4, False), (8, True), (60, False)])
def test_against_gathered_rows(tokens, cols, experts, skew):
    log(f"dispatch {tokens}x{cols} experts {experts} skew {skew}")
    x, off, src = batch(tokens + experts, tokens, cols, experts, skew)
    n = int(off[-1])
    q, s, _, _ = fb.dispatch_mxfp4_1x32(x, src)
    wq, ws = gathered(x, src)
    assert (q[:n] == wq[:n]).all() and (s[:, :n] == ws[:, :n]).all()


def test_two_streams_and_replays():
    import torch
    batches = [batch(i, 4096, 4096, 8, i == 1) for i in (1, 2)]
    ends = [int(off[-1]) for _, off, _ in batches]
    want = [gathered(x, src) for x, _, src in batches]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    outs = []
    torch.cuda.synchronize()
    for (x, _, src), g in zip(batches, graphs):
        with torch.cuda.graph(g):
            outs.append(fb.dispatch_mxfp4_1x32(x, src)[:2])
    for _ in range(5):
        got = []
        for (x, _, src), st in zip(batches, streams):
            with torch.cuda.stream(st):
                got.append(fb.dispatch_mxfp4_1x32(x, src)[:2])
        torch.cuda.synchronize()
        for out in outs:
            out[0].zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for results in (got, outs):
            for (q, s), (wq, ws), n in zip(results, want, ends):
                assert (q[:n] == wq[:n]).all() and (s[:, :n] == ws[:, :n]).all()
