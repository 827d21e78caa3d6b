"""A round as its operators are used together: peers compress their updates,
the receiver screens the records, scores every peer by the loss of given tokens
before and after its update (sl_token_logprobs on the logits of a linear
model), aggregates the peers that help and takes the outer update with momentum
and orthogonalisation (sl_muon_step).  Checked against the same round in plain
64-bit arithmetic from the same records."""
import numpy as np
import pytest
import torch

from gpu_util import note, require_gpu
from ops_reference import logprobs, muon

pytestmark = pytest.mark.gpu

ROWS, COLS, TOKENS, PEERS = 64, 512, 96, 6     # weights of 8 chunks; COLS tokens in the vocabulary


def test_scored_round(orc):
    sl = require_gpu()
    note("scored round")
    g = torch.Generator().manual_seed(5)
    n = ROWS * COLS
    theta0 = torch.randn(ROWS, COLS, generator=g) * 0.1
    inputs = torch.randn(TOKENS, ROWS, generator=g)
    targets = torch.randint(0, COLS, (TOKENS,), generator=g)
    # Peers move along the loss's gradient, the last two against it; one of the others' records is damaged.
    soft = torch.softmax(inputs @ theta0, 1)
    soft[torch.arange(TOKENS), targets] -= 1
    slope = inputs.t() @ soft / TOKENS
    payloads, scales = [], []
    for p in range(PEERS):
        noisy = slope + 0.1 * slope.std() * torch.randn(ROWS, COLS, generator=g)
        delta = (2.0 * noisy if p < PEERS - 2 else -2.0 * noisy).cuda()
        payload, scale = sl.compress(delta.flatten(), torch.zeros(n, device="cuda"))
        payloads.append(payload), scales.append(scale)
    payloads[1][3, :3] = 255                      # indices out of order
    flags = torch.empty((PEERS, n // 4096), dtype=torch.uint8, device="cuda")
    counts = torch.empty((PEERS, 4), dtype=torch.int64, device="cuda")
    smax = torch.empty(PEERS, device="cuda")
    sl.sl_peer_stats(payloads, scales, counts, smax, flags=flags)
    sound = [p for p in range(PEERS) if counts[p, 0].item() == 0]
    assert sound == [0, 2, 3, 4, 5]

    theta = theta0.cuda()
    x, t = inputs.cuda(), targets.cuda()
    before = sl.token_logprobs(x @ theta, t)[0]
    helpful, gains = [], {}
    for p in sound:
        trial = theta.clone()
        sl.sl_aggregate_apply([payloads[p]], [scales[p]], trial.view(-1))
        gains[p] = (sl.token_logprobs(x @ trial, t)[0] - before).mean().item()
        if gains[p] > 0:
            helpful.append(p)
    assert helpful == [0, 2, 3]
    out = sl.aggregate([payloads[p] for p in helpful], [scales[p] for p in helpful], n)
    momentum = torch.zeros(ROWS, COLS, device="cuda")
    sl.muon_step(theta, momentum, out.view(ROWS, COLS), lr=0.05, grad_scale=1 / len(helpful), update_scale=2.0)
    after = sl.token_logprobs(x @ theta, t, n_top=3)

    # the same in 64 bits
    records = [(payloads[p].cpu().numpy(), scales[p].cpu().numpy()) for p in range(PEERS)]
    for p in sound:
        one = torch.from_numpy(orc.aggregate([records[p][0]], [records[p][1]], n)).view(ROWS, COLS).double()
        wl = logprobs(inputs.double() @ theta0.double(), targets, 0)[0]
        wt = logprobs(inputs.double() @ (theta0.double() - one), targets, 0)[0]
        # logits of 64 products of fp32 numbers, |x theta| summing to at most about 30, each rounded: 2 * 64 * 30 * 2^-24
        assert abs(gains[p] - (wt - wl).mean().item()) < 2 * 64 * 30 * 2.0 ** -24
    total = orc.aggregate([records[p][0] for p in helpful], [records[p][1] for p in helpful], n)
    assert np.array_equal(out.cpu().numpy(), total)
    want, want_m, o, _ = muon(theta0, torch.zeros(ROWS, COLS), torch.from_numpy(total).view(ROWS, COLS), 0.05,
                              grad_scale=1 / 3, update_scale=2.0)
    # O is within 1e-5 of exact; grad_scale, the products and the result are rounded
    assert (theta.cpu().double() - want).norm() <= 0.1 * 1e-5 * o.norm() + 4 * 2.0 ** -24 * want.norm()
    assert (momentum.cpu().double() - want_m).norm() <= 4 * 2.0 ** -24 * want_m.norm()
    wl, we, wt, wi = logprobs(inputs.double() @ want, targets, 3)
    for got, w in zip((after[0], after[1], after[2]), (wl, we, wt)):
        assert (got.cpu().double() - w).abs().max() < 64 * 30 * 2.0 ** -24 * 4
    assert (after[0] - before).mean().item() > 0
