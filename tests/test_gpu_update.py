"""The matrix update (sl_orthogonalize, sl_muon_step) against its 64-bit form."""
import pytest
import torch

from gpu_util import note, require_gpu
from ops_reference import STEPS, muon, newton_schulz, newton_schulz_tolerance, relative

pytestmark = pytest.mark.gpu


def update_like(shape, seed):
    """Normal values with a lognormal factor for each row, one in a thousand 20 times as large (CPU, float32)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.randn(shape[:-1] + (1,), generator=g).exp()
    return x * (1 + 19 * (torch.rand(shape, generator=g) < 1e-3).float())


def check(got, x, products, steps=STEPS, eps=1e-7):
    """got (on the GPU) against the exact result for x, every matrix of the batch by itself."""
    got, x = got.cpu(), x.cpu()
    if x.dim() == 2:
        got, x = got[None], x[None]
    for k in range(x.shape[0]):
        exact = newton_schulz(x[k], steps, eps)
        tol = newton_schulz_tolerance(x[k], exact, products == "split", steps, eps, got.dtype)
        err = relative(got[k], exact)
        assert err <= tol, f"matrix {k} of {tuple(x.shape)}: {err:.3g} off, {tol:.3g} allowed"


SIZES = [(1, 1), (1, 7), (9, 1), (2, 300), (33, 31), (64, 64), (63, 129), (128, 192), (257, 65), (200, 1000),
         (513, 300), (640, 641)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("products", ["f16", "split"])
def test_orthogonalize_sizes(rows, cols, products):
    sl = require_gpu()
    note(f"orthogonalize {rows}x{cols} {products}")
    x = update_like((rows, cols), rows * 1000 + cols)
    out = torch.empty((rows, cols), device="cuda")
    sl.sl_orthogonalize(x.cuda(), out, products=products)
    check(out, x, products)


@pytest.mark.parametrize("x_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_orthogonalize_types(x_dtype, out_dtype):
    sl = require_gpu()
    note(f"orthogonalize {x_dtype} -> {out_dtype}")
    x = update_like((3, 90, 150), 5).to(x_dtype)
    out = sl.orthogonalize(x.cuda(), out_dtype=out_dtype)
    assert out.dtype == out_dtype
    check(out, x, "split" if out_dtype == torch.float32 else "f16")


@pytest.mark.parametrize("count,rows,cols", [(2, 1100, 1300), (9, 520, 700), (40, 130, 100), (1, 2100, 2050)])
@pytest.mark.parametrize("products", ["f16", "split"])
def test_orthogonalize_batches_and_larger_tiles(count, rows, cols, products):
    """Enough tiles that the larger ones are taken."""
    sl = require_gpu()
    note(f"orthogonalize {count}x{rows}x{cols} {products}")
    g = torch.Generator(device="cuda").manual_seed(count)
    x = torch.randn((count, rows, cols), generator=g, device="cuda")
    out = torch.empty_like(x)
    sl.sl_orthogonalize(x, out, products=products)
    some = sorted({0, count // 2, count - 1})
    for k in some:
        # the 64-bit form on the GPU: the sizes are too large for the CPU
        exact = newton_schulz(x[k])
        tol = newton_schulz_tolerance(x[k], exact, products == "split")
        err = relative(out[k], exact)
        assert err <= tol, f"matrix {k}: {err:.3g} off, {tol:.3g} allowed"


@pytest.mark.parametrize("products", ["f16", "split"])
def test_orthogonalize_thousands_of_small_matrices(products):
    sl = require_gpu()
    note(f"orthogonalize 3000 of 20x24 {products}")
    x = update_like((3000, 20, 24), 77)
    out = torch.empty(x.shape, device="cuda")
    sl.sl_orthogonalize(x.cuda(), out, products=products)
    some = [0, 1, 1499, 2999]
    check(out[some], x[some], products)
    assert out.isfinite().all()


def test_orthogonalize_strided_views_and_guards():
    """Rows and matrices of larger tensors, in and out; what lies between is left as it was."""
    sl = require_gpu()
    note("orthogonalize strided")
    big = update_like((4, 150, 333), 11).cuda()
    x = big[:, 3:120, 5:205]
    frame = torch.full((4, 160, 301), 7.0, dtype=torch.bfloat16, device="cuda")
    out = frame[:, 7:124, 1:201]
    sl.sl_orthogonalize(x, out)
    check(out, x.contiguous(), "f16")
    kept = torch.ones_like(frame, dtype=torch.bool)
    kept[:, 7:124, 1:201] = False
    assert (frame[kept] == 7.0).all()
    # every other matrix of a batch, and the same matrix for each of a batch
    y = torch.empty((2, 117, 200), device="cuda")
    sl.sl_orthogonalize(x[::2], y)
    check(y, x[::2].contiguous(), "split")
    same = x[1:2].expand(3, -1, -1)
    y = torch.empty((3, 117, 200), device="cuda")
    sl.sl_orthogonalize(same, y)
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])


@pytest.mark.parametrize("scale", [1e-38, 1e-20, 1e20, 1e36])
def test_orthogonalize_is_blind_to_scale(scale):
    """The squares of such values leave fp32's range; with eps 0 the result does not depend on the scale.  1e-38
    itself is rounded on the way in (subnormals), so the reference starts from the same rounded values."""
    sl = require_gpu()
    note(f"orthogonalize scale {scale}")
    x = update_like((70, 110), 3) * scale
    out = torch.empty((70, 110), device="cuda")
    sl.sl_orthogonalize(x.cuda(), out, eps=0.0)
    check(out, x, "split", eps=0.0)


def test_orthogonalize_zero_and_deficient():
    sl = require_gpu()
    note("orthogonalize zero and rank-deficient")
    for eps in (0.0, 1e-7):
        for dtype in (torch.float32, torch.bfloat16):
            z = sl.orthogonalize(torch.zeros((2, 70, 90), dtype=dtype, device="cuda"), eps=eps)
            assert not z.any()
    x = update_like((100, 140), 8)
    x[40:60] = 0                      # rows without an update
    x[:, 7] = 0
    x[80:] = x[:20]                   # repeated rows
    out = torch.empty(x.shape, device="cuda")
    sl.sl_orthogonalize(x.cuda(), out)
    check(out, x, "split")
    assert not out[40:60].any() and not out[:, 7].any()
    # a large eps shrinks the start
    sl.sl_orthogonalize(x.cuda(), out, eps=300.0)
    check(out, x, "split", eps=300.0)


@pytest.mark.parametrize("steps", [STEPS[:1], ((1.5, -0.5, 0.0),) * 8, ((2.0, -1.5, 0.5),) * 16,
                                   ((3.0, -3.0, 1.0), (1.875, -1.25, 0.375))])
@pytest.mark.parametrize("products", ["f16", "split"])
def test_orthogonalize_other_steps(steps, products):
    sl = require_gpu()
    note(f"orthogonalize {len(steps)} steps {products}")
    x = update_like((96, 160), 21)
    out = torch.empty(x.shape, device="cuda")
    sl.sl_orthogonalize(x.cuda(), out, coefficients=steps, products=products)
    check(out, x, products, steps)


def test_orthogonalize_repeats_bitwise_on_any_stream_and_workspace():
    sl = require_gpu()
    note("orthogonalize streams and workspaces")
    x = update_like((2, 300, 520), 4).cuda()
    first = sl.orthogonalize(x)
    need = sl.orthogonalize_workspace(300, 520, 2, "split")
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")     # NaN patterns
    guard = ws[need:].clone()
    assert torch.equal(first, sl.orthogonalize(x, workspace=ws[:need]))
    assert torch.equal(ws[need:], guard)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:                 # two calls at once, a workspace each
        outs.append(sl.orthogonalize(x, stream=s))
    with torch.cuda.stream(streams[0]):
        outs.append(sl.orthogonalize(x))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(first, o)


def test_calls_on_another_stream_use_that_streams_memory():
    """Memory that work queued on the current stream still reads is not taken for a call on another one."""
    sl = require_gpu()
    note("memory of another stream")
    x = update_like((200, 300), 4).cuda()
    logits, targets = torch.randn(64, 5000, device="cuda"), torch.arange(64, device="cuda")
    other = torch.cuda.Stream()
    calls = [(sl.orthogonalize_workspace(200, 300, 1, "split"), lambda: [sl.orthogonalize(x, stream=other)]),
             (x.numel() * 4, lambda: [sl.orthogonalize(x, stream=other.cuda_stream)]),
             (64 * 4 * 4, lambda: list(sl.token_logprobs(logits, targets, 4, stream=other)))]
    for need, call in calls:
        expected = call()
        torch.cuda.synchronize()
        kept, seen = torch.full((need,), 7, dtype=torch.uint8, device="cuda"), torch.zeros(need, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)           # some 10 ms before the copy
        seen.copy_(kept)
        del kept
        got = call()
        torch.cuda.synchronize()
        assert (seen == 7).all()
        for a, b in zip(expected, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("rows,cols,count,products", [(100, 700, 3, "f16"), (700, 100, 2, "f16"), (300, 4000, 1, "split"),
                                                      (1100, 1300, 2, "split"), (4100, 4200, 1, "f16"),
                                                      (4100, 6200, 1, "split")])
def test_workspace_contents_do_not_matter(rows, cols, count, products):
    """Every way through the products with a workspace of zeros and one of NaN patterns."""
    sl = require_gpu()
    note(f"workspace contents {count}x{rows}x{cols} {products}")
    grad = torch.randn(count, rows, cols, generator=torch.Generator().manual_seed(9)).cuda()
    results = []
    for fill in (0, 255):
        out = torch.empty_like(grad)
        need = sl.orthogonalize_workspace(rows, cols, count, products)
        sl.sl_orthogonalize(grad, out, products=products, workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
        theta, momentum = torch.ones_like(grad), torch.zeros_like(grad)
        need = sl.muon_step_workspace(rows, cols, count, products)
        sl.sl_muon_step(theta, momentum, grad, lr=0.1, products=products,
                        workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
        results.append((out, theta, momentum))
    for a, b in zip(*results):
        assert torch.equal(a, b) and a.isfinite().all()


def run_muon(sl, theta, momentum, grad, **kw):
    t, m = theta.cuda(), momentum.cuda()
    sl.muon_step(t, m, grad.cuda(), **kw)
    return t.cpu(), m.cpu()


@pytest.mark.parametrize("theta_dtype,grad_dtype,products",
                         [(torch.float32, torch.float32, "split"), (torch.float32, torch.bfloat16, "f16"),
                          (torch.bfloat16, torch.bfloat16, "f16"), (torch.bfloat16, torch.float32, "split")])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("count,rows,cols", [(1, 130, 67), (3, 65, 200), (2, 33, 33)])
def test_muon_step(theta_dtype, grad_dtype, products, nesterov, count, rows, cols):
    sl = require_gpu()
    note(f"muon {count}x{rows}x{cols} {theta_dtype} {grad_dtype} {products} nesterov={nesterov}")
    theta = (torch.randn(count, rows, cols, generator=torch.Generator().manual_seed(1)) * 0.02).to(theta_dtype)
    momentum, grad = update_like((count, rows, cols), 2), update_like((count, rows, cols), 3).to(grad_dtype)
    kw = dict(lr=0.02, grad_scale=1 / 3, decay=0.9, nesterov=nesterov, weight_decay=0.1, update_scale=1.7)
    t, m = run_muon(sl, theta, momentum, grad, products=products, **kw)
    for k in range(count):
        want_t, want_m, o, u = muon(theta[k], momentum[k], grad[k], **kw)
        # grad_scale, decay and the product g are rounded to fp32, then one fused multiply-add: each value is
        # off by at most (2^-24) (2 |g| + 2 |decay m| + |m'|) up to second order
        g = grad[k].double().abs() / 3
        bound = 2.0 ** -24 * (2 * g + 2 * 0.9 * momentum[k].double().abs() + want_m.abs()) * 1.01
        assert ((m[k].double() - want_m).abs() <= bound).all()
        # O's error, then the rounding of keep, move, their products and the result
        tol = newton_schulz_tolerance(u, o, products == "split")
        off = (t[k].double() - want_t).norm().item()
        move = 0.02 * 1.7 * o.norm().item()
        rounding = (torch.finfo(theta_dtype).eps / 2 + 3 * 2.0 ** -24) * want_t.norm().item() + 3 * 2.0 ** -24 * move
        # u itself is off by a few 2^-24 of the momentum's terms, stretched by the steps as X's own rounding is
        assert off <= move * (tol + 64 * 2.0 ** -24) + rounding


@pytest.mark.parametrize("rows,cols", [(1800, 2701), (2703, 1799)])
def test_muon_step_of_large_matrices_by_their_gram_matrix(rows, cols):
    """Split operands, large, one side 1.5 times the other: three steps at a time on the Gram matrix.  An error of
    22 bits in R is stretched, where R's eigenvalues are smallest, by the square of a step's largest factor 3.4445
    for each of the two steps that follow: 141 * 2^-22 / 3 = 1.1e-5 if every eigenvalue were that small (a third of
    them, say), in each of the two runs of steps."""
    sl = require_gpu()
    note(f"muon by gram {rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(rows)
    grad = torch.randn((4, rows, cols), generator=g, device="cuda")
    grad *= torch.randn((4, rows, 1), generator=g, device="cuda").exp()
    theta, momentum = torch.zeros_like(grad), torch.zeros_like(grad)
    sl.muon_step(theta, momentum, grad, lr=1.0, nesterov=False, products="split")
    assert torch.equal(momentum, grad)
    for k in (0, 3):
        err = relative(-theta[k], newton_schulz(grad[k]))
        assert err <= 2 * 1.1e-5, err
    # four steps end in a run of one; momentum is momentum * 0.95 + grad by now
    theta.zero_()
    sl.muon_step(theta, momentum, grad, lr=1.0, nesterov=False, products="split", coefficients=STEPS[:4])
    err = relative(-theta[1], newton_schulz(momentum[1], STEPS[:4]))
    assert err <= 2 * 1.1e-5, err
    # steps that let Q grow past what fp16 pairs should carry take the other way
    steps = ((3.7, -5.3, 2.2), (8.0, -14.0, 6.0), (9.0, -8.0, 1.2))
    theta.zero_()
    sl.muon_step(theta, momentum, grad, lr=1.0, nesterov=False, products="split", coefficients=steps)
    want = newton_schulz(momentum[2], steps)
    tol = newton_schulz_tolerance(momentum[2], want, True, steps)
    assert relative(-theta[2], want) <= tol


@pytest.mark.parametrize("count,rows,cols", [(1, 70, 900), (3, 900, 70), (22, 190, 400), (1, 520, 4300), (2, 2210, 1000)])
def test_split_products_of_long_matrices_by_their_gram_matrix(count, rows, cols):
    """64 x 64 and 128 x 128 tiles, one side at least twice the other.  The bound is that of the other way: an error of
    22 bits in R, stretched by at most 141, is at most 1.1e-5 for each run of steps were all eigenvalues the smallest."""
    sl = require_gpu()
    note(f"orthogonalize by gram {count}x{rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn((count, rows, cols), generator=g, device="cuda")
    x *= torch.randn((count, rows, 1), generator=g, device="cuda").exp()
    out = sl.orthogonalize(x)
    theta, momentum = torch.zeros_like(x), torch.zeros_like(x)
    sl.muon_step(theta, momentum, x, lr=1.0, nesterov=False)
    assert torch.equal(theta, -out) and torch.equal(momentum, x)
    for k in {0, count - 1}:
        err = relative(out[k], newton_schulz(x[k]))
        assert err <= 2 * 1.1e-5, err
    for n_steps in (1, 3, 4):
        out = sl.orthogonalize(x, coefficients=STEPS[:n_steps])
        err = relative(out[count - 1], newton_schulz(x[count - 1], STEPS[:n_steps]))
        assert err <= 2 * 1.1e-5, (n_steps, err)
    zero = sl.orthogonalize(torch.zeros_like(x))
    assert not zero.any()


@pytest.mark.parametrize("rows,cols", [(96, 64), (80, 64), (140, 128), (50, 40), (24, 16), (64, 96), (256, 64), (520, 64)])
def test_plain_products_of_tall_matrices_with_uneven_rows(rows, cols):
    """Small singular values, which roundings of the Gram matrix would drown."""
    sl = require_gpu()
    note(f"plain products, uneven rows {rows}x{cols}")
    x = update_like((12, rows, cols), 7 * rows + cols)
    check(sl.orthogonalize(x.cuda(), products="f16"), x, "f16")


@pytest.mark.parametrize("count,rows,cols", [(1, 600, 9000), (1, 1300, 2800), (1, 8192, 1024), (1, 520, 4300)])
def test_steep_steps_of_long_matrices_stay_in_their_workspace(count, rows, cols):
    """Sizes that go by the Gram matrix, with coefficients that do not: on a workspace of exactly the stated size."""
    sl = require_gpu()
    note(f"steep steps {count}x{rows}x{cols}")
    steps = ((3.7, -5.3, 2.2), (8.0, -14.0, 6.0), (9.0, -8.0, 1.2))
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn((count, rows, cols), generator=g, device="cuda")
    need = sl.orthogonalize_workspace(rows, cols, count, "split")
    whole = torch.full((need + (64 << 20),), 170, dtype=torch.uint8, device="cuda")
    for coefficients in (steps, STEPS):
        out = torch.empty_like(x)
        sl.sl_orthogonalize(x, out, coefficients=coefficients, workspace=whole[:need])
        assert (whole[need:] == 170).all()
        want = newton_schulz(x[0], coefficients)
        # the steep steps' bound, as the other way has it; that of the Gram matrix's for the usual ones
        tol = newton_schulz_tolerance(x[0], want, True, coefficients) if coefficients is steps else 2 * 1.1e-5
        assert relative(out[0], want) <= tol


def test_muon_step_is_the_composition():
    """theta's move is what sl_orthogonalize gives for the same u: bitwise with keep 1 and move 1 from zero weights."""
    sl = require_gpu()
    note("muon composition")
    grad, momentum = update_like((2, 140, 90), 5).cuda(), update_like((2, 140, 90), 6).cuda()
    theta = torch.zeros((2, 140, 90), device="cuda")
    before = momentum.clone()
    sl.muon_step(theta, momentum, grad, lr=1.0, decay=0.5, nesterov=False)
    assert torch.equal(momentum, torch.add(grad, before, alpha=0.5))   # 0.5 m is exact: one rounding either way
    assert torch.equal(theta, -sl.orthogonalize(momentum))


def test_muon_step_zero_sizes_and_zero_gradient():
    sl = require_gpu()
    note("muon zero")
    for shape in ((0, 5), (5, 0), (0, 4, 4)):
        z = torch.zeros(shape, device="cuda")
        sl.muon_step(z, z.clone(), z.clone(), lr=1.0)
        assert sl.orthogonalize(z).shape == z.shape
    theta = torch.ones((40, 50), device="cuda")
    momentum = torch.zeros_like(theta)
    sl.muon_step(theta, momentum, torch.zeros_like(theta), lr=0.5, weight_decay=0.5)
    assert (theta == 0.75).all() and not momentum.any()


def test_updates_in_a_graph():
    """A captured round of updates, replayed with eager work in between, against the eager calls."""
    sl = require_gpu()
    note("muon in a graph")
    theta0 = (torch.randn(130, 200, generator=torch.Generator().manual_seed(1)) * 0.02).cuda()
    momentum0, grad = update_like((130, 200), 2).cuda(), update_like((130, 200), 3).cuda()
    ws = torch.empty(sl.muon_step_workspace(130, 200, 1, "split"), dtype=torch.uint8, device="cuda")
    theta, momentum = theta0.clone(), momentum0.clone()
    out = torch.empty_like(theta)
    sl.muon_step(theta, momentum, grad, lr=0.02, workspace=ws)        # warm up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sl.muon_step(theta, momentum, grad, lr=0.02, workspace=ws)
        sl.sl_orthogonalize(theta, out, workspace=ws)
    theta.copy_(theta0), momentum.copy_(momentum0)
    t, m = theta0.clone(), momentum0.clone()
    for k in range(4):
        graph.replay()
        torch.cuda.synchronize()
        sl.muon_step(t, m, grad, lr=0.02)
        assert torch.equal(theta, t) and torch.equal(momentum, m)
        assert torch.equal(out, sl.orthogonalize(t))
        grad.mul_(-0.7)
        torch.cuda.synchronize()
