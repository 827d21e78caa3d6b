"""sl_token_logprobs against its 64-bit form."""
import math

import pytest
import torch

from gpu_util import note, require_gpu
from ops_reference import logprobs

pytestmark = pytest.mark.gpu
INF = float("inf")


def compare(got, want, x, banned_too=False):
    """logprob, entropy and top_logprob within fp32's reach, the indices equal.

    x - m is exact up to half a step of |x - m|; exp and the sum of at most 2^22
    terms (16 in a row per lane and tile, tiles in a row, then a tree) leave
    log s off by at most about 200 * 2^-24 even if every rounding of a lane's
    sum went one way (262208 tokens: 64 tiles of 16 adds over 64 lanes' tree
    would be 1100 * 2^-24 at worst, their random sum 33 * 2^-24); the exponents
    (x - m) log2 e are off by 1.5 * 2^-24 |x - m|, which counts weighted by
    exp(x - m) |x - m| <= 0.37."""
    logprob, entropy, top_logprob, top_index = (t.cpu() if t is not None else None for t in got)
    wl, we, wt, wi = want
    for g, w in ((logprob, wl), (entropy, we), (top_logprob, wt)):
        if g is None:
            continue
        assert torch.equal(g.isnan(), w.isnan())
        assert torch.equal(g == -INF, w == -INF)
        ok = w.isfinite()
        assert g[ok].isfinite().all()
        off = (g[ok].double() - w[ok]).abs()
        assert (off <= 2.0 ** -24 * (200 + 4 * w[ok].abs())).all(), off.max()
    if top_index is not None:
        assert torch.equal(top_index, wi)


def run(sl, logits, targets, n_top, **kw):
    return sl.token_logprobs(logits.cuda(), targets.cuda(), n_top, **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,vocab,n_top", [(1, 1, 1), (3, 2, 5), (1, 5000, 20), (5, 1023, 32), (4, 1024, 7),
                                              (7, 1025, 1), (2, 33000, 32), (40, 2049, 3), (1, 70001, 0), (0, 10, 2)])
def test_sizes(dtype, rows, vocab, n_top):
    sl = require_gpu()
    note(f"logprobs {rows}x{vocab} {dtype} top {n_top}")
    g = torch.Generator().manual_seed(rows * 7 + vocab)
    x = (torch.randn(rows, vocab, generator=g) * 3).to(dtype)
    t = torch.randint(0, vocab, (rows,), generator=g)
    compare(run(sl, x, t, n_top), logprobs(x, t, n_top), x)


def test_large_vocabulary_many_rows():
    sl = require_gpu()
    note("logprobs 70 x 262208 and 2 x 4194304")
    for rows, vocab, dtype in ((70, 262208, torch.bfloat16), (2, 1 << 22, torch.bfloat16), (1, 262143, torch.float32)):
        g = torch.Generator().manual_seed(rows)
        x = (torch.randn(rows, vocab, generator=g) * 2).to(dtype)
        t = torch.randint(0, vocab, (rows,), generator=g)
        compare(run(sl, x, t, 20), logprobs(x, t, 20), x)


def test_more_rows_than_a_grid_holds():
    sl = require_gpu()
    note("logprobs 70000 x 50")
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(70000, 50, generator=g) * 3).bfloat16()
    t = torch.randint(0, 50, (70000,), generator=g)
    got = run(sl, x, t, 2)
    some = torch.cat([torch.arange(40), torch.arange(65500, 65600), torch.arange(69960, 70000)])
    compare([o.cpu()[some] for o in got], logprobs(x[some], t[some], 2), x)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_ties_go_to_the_lower_token(dtype):
    sl = require_gpu()
    note(f"logprobs ties {dtype}")
    g = torch.Generator().manual_seed(9)
    vocab = 5000
    x = torch.randint(-2, 3, (12, vocab), generator=g).to(dtype)
    x[0] = 0                                    # every token equal
    x[1] = -0.0
    x[1, 4001] = 0.0                            # equal to -0
    x[2] = -1
    x[2, [17, 1023, 1024, 4999]] = 1            # ties across tiles
    x[3] = torch.arange(vocab).to(dtype) / 64   # ascending: the last tokens
    x[4] = -torch.arange(vocab).to(dtype) / 64
    x[5] = torch.finfo(dtype).min               # uniform at the type's lowest value
    x[6] = torch.finfo(dtype).min
    x[6, 3000] = 0
    x[7] = torch.finfo(dtype).max
    t = torch.randint(0, vocab, (12,), generator=g)
    for n_top in (1, 2, 32):
        compare(run(sl, x, t, n_top), logprobs(x, t, n_top), x)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_banned_tokens_and_bad_rows(dtype):
    sl = require_gpu()
    note(f"logprobs banned {dtype}")
    g = torch.Generator().manual_seed(10)
    vocab = 3001
    x = (torch.randn(10, vocab, generator=g) * 2).to(dtype)
    x[0] = -INF                                 # nothing is left
    x[1, :2999] = -INF                          # two tokens left
    x[2, 5:] = -INF
    x[3] = -INF
    x[3, 1500] = 4                              # one token
    x[4, 77] = float("nan")
    x[5, 2999] = INF
    x[6] = -INF
    x[6, 10] = float("nan")
    x[7, ::2] = -INF
    x[8, 100] = 300                             # all but certain
    t = torch.tensor([4, 3000, 2, 1500, 3, 5, 10, 1, 100, 50])
    compare(run(sl, x, t, 6), logprobs(x, t, 6), x)
    t = torch.tensor([-100, vocab, 9, 0, -1, vocab + 7, -1, 2, 101, -(1 << 40)])    # no token, and a banned one
    compare(run(sl, x, t, 0), logprobs(x, t, 0), x)


def test_strided_rows_of_every_alignment_and_partial_outputs():
    sl = require_gpu()
    note("logprobs strided")
    g = torch.Generator().manual_seed(12)
    for dtype in (torch.bfloat16, torch.float32):
        big = (torch.randn(9, 4111, generator=g) * 2).to(dtype).cuda()
        big[:, :3] = 50                          # neighbours that must not count
        big[:, 3003:] = 60
        x = big[:, 3:3003]
        t = torch.randint(0, 3000, (9,), generator=g)
        want = logprobs(x, t, 4)
        compare(sl.token_logprobs(x, t.cuda(), 4), want, x)
        one = torch.empty(9, device="cuda")
        sl.sl_token_logprobs(x, t.cuda(), one, None)
        compare((one, None, None, None), want, x)
        sl.sl_token_logprobs(x, None, None, one)
        compare((want[0].float(), one, None, None), want, x)


def test_repeats_bitwise_and_streams():
    sl = require_gpu()
    note("logprobs streams")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((5, 40000), generator=g, device="cuda").bfloat16()
    t = torch.randint(0, 40000, (5,), generator=g, device="cuda")
    first = sl.token_logprobs(x, t, 9)
    need = sl.token_logprobs_workspace(5, 40000, torch.bfloat16, 9)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [sl.token_logprobs(x, t, 9, workspace=ws[:need])]
    outs += [sl.token_logprobs(x, t, 9, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert (ws[need:] == 255).all()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(first, o))


def test_in_a_graph():
    sl = require_gpu()
    note("logprobs in a graph")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((3, 20000), generator=g, device="cuda")
    t = torch.randint(0, 20000, (3,), generator=g, device="cuda")
    lp, ent = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    tl, ti = torch.empty((3, 5), device="cuda"), torch.empty((3, 5), dtype=torch.int32, device="cuda")
    ws = torch.empty(sl.token_logprobs_workspace(3, 20000, torch.float32, 5), dtype=torch.uint8, device="cuda")
    sl.sl_token_logprobs(x, t, lp, ent, tl, ti, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sl.sl_token_logprobs(x, t, lp, ent, tl, ti, ws)
    for k in range(3):
        x.mul_(-1.3)
        for o in (lp, ent, tl):
            o.fill_(math.nan)
        ti.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((lp, ent, tl, ti), sl.token_logprobs(x, t, 5)):
            assert torch.equal(a, b)
