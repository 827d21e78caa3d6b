"""Cases of the matrix update and token score operators, in their plain form and as the library's calls.

Three operators, each with its plain form in elementary torch operations:

  orthogonalize   Newton-Schulz orthogonalisation of an update: X <- x / (|x|_F + eps), then for each
                  (a, b, c): A = X X^T, X <- a X + (b A + c A A) X
  muon_step       momentum, orthogonalisation and weight update of one weight matrix (or several equal ones):
                  g = grad_scale * grad, m <- decay * m + g, u = g + decay * m,
                  theta <- theta * (1 - lr * weight_decay) - lr * update_scale * orthogonalize(u)
  token_logprobs  log probabilities of given tokens with the distribution's entropy and its n_top likeliest
                  tokens (ties go to the lower token), as a score of received updates needs them

`own` is set from outside: with it, run() calls the library; without it, the plain forms.
"""
import math

import torch

own = False

# The quintic of the orthogonalisation, used for each of five steps.
COEFFICIENTS = ((3.4445, -4.7750, 2.0315),) * 5
EPS = 1e-7
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def listed():
    return [
        # One small matrix, where the call's latency counts.
        {"name": "orth_small", "op": "orthogonalize", "count": 1, "rows": 128, "cols": 192,
         "dtype": "bfloat16", "out": "bfloat16"},
        # The eight key/value heads of a K projection, each head's 8192 x 128 block orthogonalised by itself.
        {"name": "orth_kv_heads", "op": "orthogonalize", "count": 8, "rows": 8192, "cols": 128,
         "dtype": "bfloat16", "out": "bfloat16"},
        # Ragged sizes, float32 in and out.
        {"name": "orth_ragged", "op": "orthogonalize", "count": 3, "rows": 1000, "cols": 2731,
         "dtype": "float32", "out": "float32"},
        # An attention projection of the 8192-wide model, 16-bit result.
        {"name": "orth_attention", "op": "orthogonalize", "count": 1, "rows": 8192, "cols": 8192,
         "dtype": "bfloat16", "out": "bfloat16"},
        # Small weight matrices of one shape, inner steps on 16-bit weights.
        {"name": "muon_small", "op": "muon_step", "count": 6, "rows": 333, "cols": 517, "theta": "bfloat16",
         "grad": "bfloat16", "nesterov": True, "grad_scale": 1.0, "lr": 0.02, "weight_decay": 0.1},
        # The K projection's outer update: the sum of 24 peers' updates as gradient, float32 weights.
        {"name": "muon_kv_outer", "op": "muon_step", "count": 1, "rows": 8192, "cols": 1024, "theta": "float32",
         "grad": "float32", "nesterov": True, "grad_scale": 1.0 / 24, "lr": 0.004, "weight_decay": 0.0},
        # An attention projection's inner step on 16-bit weights.
        {"name": "muon_attention", "op": "muon_step", "count": 1, "rows": 8192, "cols": 8192, "theta": "bfloat16",
         "grad": "bfloat16", "nesterov": True, "grad_scale": 1.0, "lr": 0.002, "weight_decay": 0.1},
        # The outer update of an MLP matrix, the largest matrix of the 8192-wide model.
        {"name": "muon_mlp_outer", "op": "muon_step", "count": 1, "rows": 8192, "cols": 28672, "theta": "float32",
         "grad": "float32", "nesterov": False, "grad_scale": 1.0 / 24, "lr": 0.004, "weight_decay": 0.0},
        # One position of the 262,208-token vocabulary.
        {"name": "logprob_one", "op": "token_logprobs", "rows": 1, "vocab": 262208, "dtype": "bfloat16",
         "n_top": 20, "banned": 0.0},
        # A short text, float32 logits of an odd vocabulary, some tokens banned.
        {"name": "logprob_ragged", "op": "token_logprobs", "rows": 157, "vocab": 100003, "dtype": "float32",
         "n_top": 8, "banned": 0.01},
        # A scoring batch: losses and entropies alone.
        {"name": "logprob_score", "op": "token_logprobs", "rows": 1024, "vocab": 262208, "dtype": "bfloat16",
         "n_top": 0, "banned": 0.0},
        # A long text with its likeliest alternatives.
        {"name": "logprob_long", "op": "token_logprobs", "rows": 4096, "vocab": 262208, "dtype": "bfloat16",
         "n_top": 5, "banned": 0.0},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49))))))


def draw(rng):
    op = rng.choice(("orthogonalize", "muon_step", "token_logprobs"))
    if op == "token_logprobs":
        vocab = _spread(rng, 1000, 262208)
        rows = _spread(rng, 1, min(8192, 4096 * 262208 // vocab))
        dtype = rng.choice(("bfloat16", "float16", "float32"))
        return {"op": op, "rows": rows if dtype != "float32" else (rows + 1) // 2, "vocab": vocab, "dtype": dtype,
                "n_top": rng.choice((0, 1, 5, 20, 32)), "banned": rng.choice((0.0, 0.01, 0.5))}
    rows, cols = _spread(rng, 16, 8192), _spread(rng, 16, 8192)
    count = _spread(rng, 1, max(1, min(32, (1 << 23) // (rows * cols))))
    if op == "orthogonalize":
        return {"op": op, "count": count, "rows": rows, "cols": cols, "dtype": rng.choice(("float32", "bfloat16")),
                "out": rng.choice(("float32", "bfloat16"))}
    theta, outer = rng.choice(("float32", "bfloat16")), rng.random() < 0.5
    return {"op": op, "count": count, "rows": rows, "cols": cols, "theta": theta,
            "grad": "float32" if outer else rng.choice(("float32", "bfloat16")), "nesterov": rng.random() < 0.5,
            "grad_scale": 1.0 / 24 if outer else 1.0, "lr": rng.choice((0.002, 0.004, 0.02)),
            "weight_decay": rng.choice((0.0, 0.1))}


def _update(shape, gen):
    """Values as an update has them: normal, a lognormal factor for each row, one in a thousand 20 times as large."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.randn(shape[:-1] + (1,), generator=gen, device="cuda").exp_()
    return x.mul_((torch.rand(shape, generator=gen, device="cuda") < 1e-3).float().mul_(19).add_(1))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] == "token_logprobs":
        shape = (case["rows"], case["vocab"])
        logits = torch.randn(shape, generator=gen, device="cuda").mul_(2.5)
        targets = torch.randint(0, case["vocab"], (case["rows"],), generator=gen, device="cuda")
        # Most text is predicted well: the target's logit stands out in two rows of three.
        lift = torch.rand(case["rows"], generator=gen, device="cuda")
        rows = torch.arange(case["rows"], device="cuda")
        logits[rows, targets] += torch.where(lift < 0.67, 16 * lift, 0.0)
        if case["banned"]:
            banned = torch.rand(case["vocab"], generator=gen, device="cuda") < case["banned"]
            logits[:, banned] = -math.inf
        return {"case": case, "logits": logits.to(DTYPES[case["dtype"]]), "targets": targets}
    shape = (case["count"], case["rows"], case["cols"])
    if case["op"] == "orthogonalize":
        return {"case": case, "x": _update(shape, gen).to(DTYPES[case["dtype"]])}
    return {
        "case": case,
        "theta": torch.randn(shape, generator=gen, device="cuda").mul_(0.02).to(DTYPES[case["theta"]]),
        "momentum": _update(shape, gen).mul_(2 * case["grad_scale"]),
        "grad": _update(shape, gen).to(DTYPES[case["grad"]]),
        # One choice of scale in use: the update's root mean square is 0.2 whatever the shape.
        "update_scale": 0.2 * math.sqrt(max(case["rows"], case["cols"])),
    }


def _orthogonalize(x):
    """The plain form, float32 [count, rows, cols]; the norm in 64 bits, since it scales every step."""
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    norm = x.double().square().sum((-2, -1), keepdim=True).sqrt()
    x = (x / (norm + EPS)).float()
    for a, b, c in COEFFICIENTS:
        gram = x @ x.mT.contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.mT if tall else x


def _muon_step(state):
    case, theta, momentum = state["case"], state["theta"], state["momentum"]
    grad = state["grad"].float() * case["grad_scale"]
    momentum.mul_(0.95).add_(grad)
    update = grad + 0.95 * momentum if case["nesterov"] else momentum
    moved = theta.float() * (1 - case["lr"] * case["weight_decay"])
    theta.copy_(moved - case["lr"] * state["update_scale"] * _orthogonalize(update))
    return {"theta": theta, "momentum": momentum}


def _token_logprobs(logits, targets, n_top):
    x = logits.float()
    rows = torch.arange(x.shape[0], device=x.device)
    top = x.amax(1, keepdim=True)
    shifted = x - top
    weight = shifted.exp()
    total = weight.sum(1)
    log_total = total.log()
    logprob = shifted[rows, targets] - log_total
    entropy = log_total - torch.where(weight > 0, weight * shifted, 0.0).sum(1) / total
    if not n_top:
        return {"logprob": logprob, "entropy": entropy}
    # One 64-bit key for each token, larger for a larger logit and then for a lower token.
    bits = (x + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32
    key |= 0xFFFFFFFF - torch.arange(x.shape[1], device=x.device)
    index = 0xFFFFFFFF - (key.topk(n_top, 1).values & 0xFFFFFFFF)
    top_logprob = shifted.gather(1, index) - log_total[:, None]
    index = torch.where(top_logprob == -math.inf, -1, index).int()
    return {"logprob": logprob, "entropy": entropy, "top_logprob": top_logprob, "top_index": index}


def run(state):
    case = state["case"]
    if own:
        import communication_efficient_distributed_amd as sl
        if case["op"] == "orthogonalize":
            return sl.orthogonalize(state["x"], out_dtype=DTYPES[case["out"]], coefficients=COEFFICIENTS, eps=EPS)
        if case["op"] == "muon_step":
            sl.muon_step(state["theta"], state["momentum"], state["grad"], case["lr"], grad_scale=case["grad_scale"],
                         decay=0.95, nesterov=case["nesterov"], weight_decay=case["weight_decay"],
                         update_scale=state["update_scale"], coefficients=COEFFICIENTS, eps=EPS)
            return {"theta": state["theta"], "momentum": state["momentum"]}
        logprob, entropy, top_logprob, top_index = sl.token_logprobs(state["logits"], state["targets"], case["n_top"])
        if not case["n_top"]:
            return {"logprob": logprob, "entropy": entropy}
        return {"logprob": logprob, "entropy": entropy, "top_logprob": top_logprob, "top_index": top_index}
    if case["op"] == "orthogonalize":
        return _orthogonalize(state["x"].float()).to(DTYPES[case["out"]])
    if case["op"] == "muon_step":
        return _muon_step(state)
    return _token_logprobs(state["logits"], state["targets"], case["n_top"])


def work(case):
    """Inputs read once and outputs written once; for the orthogonalisation, five steps of the symmetric products
    X X^T and A A, half of each, and of the full product with X (2 operations for each multiplication)."""
    size = {"float32": 4, "bfloat16": 2, "float16": 2}
    if case["op"] == "token_logprobs":
        values = case["rows"] * case["vocab"]
        return {"bytes": values * size[case["dtype"]] + case["rows"] * (8 + 8 + 8 * case["n_top"]),
                "flops": 5 * values}
    values = case["count"] * case["rows"] * case["cols"]
    short, long = sorted((case["rows"], case["cols"]))
    flops = len(COEFFICIENTS) * case["count"] * (3 * short * short * long + short ** 3)
    if case["op"] == "orthogonalize":
        return {"bytes": values * (size[case["dtype"]] + size[case["out"]]), "flops": flops}
    return {"bytes": values * (2 * size[case["theta"]] + 2 * 4 + size[case["grad"]]), "flops": flops}


def _exact_orthogonalize(x):
    """One float64 matrix: the steps as polynomials of the smaller Gram matrix, applied from its side."""
    x = x / (torch.linalg.vector_norm(x) + EPS)
    left = x.shape[0] <= x.shape[1]
    for a, b, c in COEFFICIENTS:
        gram = x.matmul(x.t()) if left else x.t().matmul(x)
        poly = gram.matmul(gram).mul_(c).add_(gram, alpha=b)
        poly.diagonal().add_(a)
        x = poly.matmul(x) if left else x.matmul(poly)
    return x


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "orthogonalize":
        return torch.stack([_exact_orthogonalize(x.double()) for x in state["x"]])
    if case["op"] == "muon_step":
        theta, momentum = state["theta"].double(), state["momentum"].double()
        for k in range(case["count"]):
            grad = state["grad"][k].double() * case["grad_scale"]
            momentum[k] = grad + 0.95 * momentum[k]
            update = momentum[k] * 0.95 + grad if case["nesterov"] else momentum[k]
            theta[k] -= case["lr"] * (case["weight_decay"] * theta[k]
                                      + state["update_scale"] * _exact_orthogonalize(update))
        return {"theta": theta, "momentum": momentum}
    n_top, out = case["n_top"], {"logprob": [], "entropy": [], "top_logprob": []}
    for logits, target in zip(state["logits"].split(256), state["targets"].split(256)):
        logp = torch.log_softmax(logits.double(), 1)
        out["logprob"].append(logp.gather(1, target[:, None])[:, 0])
        out["entropy"].append(-(logp.exp() * logp.clamp_min(-1e4)).sum(1))
        out["top_logprob"].append(logp.sort(1, descending=True).values[:, :n_top] if n_top else logp[:, :0])
    out = {k: torch.cat(v) for k, v in out.items()}
    if not n_top:
        del out["top_logprob"]
        return out
    return {**out, "top_index": None}
