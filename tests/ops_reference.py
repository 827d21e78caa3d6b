"""Plain 64-bit forms of the operators in include/sparseloco_ops.h, for the
tests: written from the formulas, without the library."""
import torch

STEPS = ((3.4445, -4.7750, 2.0315),) * 5


def _rounded(v, bits):
    """v as fp16 holds it (bits 11), or as the sum of two fp16 values (22), or as it is (None)."""
    if bits is None:
        return v
    hi = v.float().half()
    out = hi.double()
    return out if bits == 11 else out + (v.float() - hi.float()).half().double()


def newton_schulz(x, steps=STEPS, eps=1e-7, bits=None):
    """The exact orthogonalisation of one matrix in fp64 (bits None).  With
    bits, the same with every operand rounded as the library's products round
    it (X times 2^13, A times 2^12 and B times 2^11 without their diagonals),
    all else in fp64: its distance from the exact result says what those
    roundings cost."""
    x = x.double()
    if x.shape[0] > x.shape[1]:
        return newton_schulz(x.t(), steps, eps, bits).t()
    norm = x.square().sum().sqrt() + eps
    x = x / norm if norm > 0 else torch.zeros_like(x)

    def off_diagonal(m, scale):
        d = torch.diag(m.diagonal())
        return _rounded((m - d) * scale, bits) / scale + d

    x = _rounded(x * 2 ** 13, bits) / 2 ** 13
    for k, (a, b, c) in enumerate(steps):
        gram = off_diagonal(x @ x.t(), 2 ** 12)
        poly = off_diagonal(b * gram + c * (gram @ gram), 2 ** 11)
        x = a * x + poly @ x
        if k + 1 < len(steps):
            x = _rounded(x * 2 ** 13, bits) / 2 ** 13
    return x


def relative(got, want):
    want = want.double()
    norm = want.norm().item()
    off = (got.double() - want).norm().item()
    return off / norm if norm else off


def newton_schulz_tolerance(x, exact, split, steps=STEPS, eps=1e-7, out_dtype=torch.float32):
    """How far (2-norm over 2-norm) the library's result may be from exact.

    The roundings of the operands cost what the fp64 model with those roundings
    shows, on other sums of the same inputs; 3 times that covers the difference
    between one set of roundings and another.  The fp32 sums add at most
    2^-24 for each of the K / 16 partial sums of a matrix instruction (three
    times as many for split operands), at random signs sqrt of that number,
    relative to the entries' root mean square, in each of the three products of
    each step; a step stretches an error by at most 3.5, and after the steps of
    most growth X itself has grown as much, so the relative error of the last
    product counts once and that of the others at most about as often as there
    are steps: 3 * steps * sqrt(3 K / 16) * 2^-24.  The output's rounding adds
    half a step at most."""
    model = relative(newton_schulz(x, steps, eps, 22 if split else 11), exact)
    k = max(x.shape)
    sums = 3 * len(steps) * (3 * k / 16 + 1) ** 0.5 * 2.0 ** -24
    return 3 * model + sums + torch.finfo(out_dtype).eps / 2


def muon(theta, momentum, grad, lr, grad_scale=1.0, decay=0.95, nesterov=True, weight_decay=0.0, update_scale=1.0,
         steps=STEPS, eps=1e-7):
    """(theta, momentum, update) after one step, fp64."""
    g = grad.double() * grad_scale
    m = decay * momentum.double() + g
    u = g + decay * m if nesterov else m
    o = newton_schulz(u, steps, eps)
    return theta.double() * (1 - lr * weight_decay) - lr * update_scale * o, m, o, u


def logprobs(logits, targets, n_top):
    """(logprob, entropy, top_logprob, top_index) in fp64 by sl_token_logprobs' definition."""
    x = logits.double().cpu()
    rows, vocab = x.shape
    bad = (x.isnan() | (x == float("inf"))).any(1)
    empty = (x == -float("inf")).all(1)
    safe = torch.where((bad | empty)[:, None], torch.zeros_like(x), x)
    safe = safe - safe.amax(1, keepdim=True)  # values near the type's largest would swallow lse
    lse = safe.logsumexp(1)
    logp = safe - lse[:, None]
    plogp = torch.where(logp == -float("inf"), torch.zeros_like(logp), logp.exp() * logp)
    entropy = torch.where(empty, 0.0, -plogp.sum(1))
    entropy[bad] = float("nan")
    t = targets.cpu()
    inside = (t >= 0) & (t < vocab)
    logprob = logp.gather(1, t.clamp(0, vocab - 1)[:, None])[:, 0]
    logprob[empty] = -float("inf")
    logprob[bad] = float("nan")
    logprob[~inside] = 0.0
    top_logprob = torch.full((rows, n_top), -float("inf"), dtype=torch.float64)
    top_index = torch.full((rows, n_top), -1, dtype=torch.int32)
    for r in range(rows):
        if bad[r]:
            top_logprob[r] = float("nan")
        elif n_top and not empty[r]:
            order = torch.sort(x[r] + 0.0, descending=True, stable=True).indices[:n_top]
            order = order[x[r][order] > -float("inf")]
            top_index[r, :len(order)] = order.int()
            top_logprob[r, :len(order)] = logp[r][order]
    return logprob, entropy, top_logprob, top_index
