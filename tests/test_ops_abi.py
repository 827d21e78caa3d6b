"""Host-side tests of include/sparseloco_ops.h: exports, refusals before
anything reaches the GPU, workspace sizes, and the kernels' resources.  Pointer
arguments are fake addresses; argument checks never dereference them."""
import ctypes
import importlib.util
import math
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sparseloco_ops.h")
SL_OK, SL_ERR_INVALID_ARG, SL_ERR_SHAPE, SL_ERR_ALIGN = 0, 1, 2, 3
A = 1 << 28
X, OUT, M, WS, T, LP, EN, TL, TI = (A * k for k in range(1, 10))
QUINTIC = (3.4445, -4.7750, 2.0315)
nan, inf = math.nan, math.inf


@pytest.fixture(scope="module")
def lib():
    from communication_efficient_distributed_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from communication_efficient_distributed_amd import _build
        _build.build_library()
    return _lib.load()


def test_library_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(sl_[a-z_]+)\s*\(", text))
    assert {"sl_orthogonalize", "sl_muon_step", "sl_token_logprobs"} <= names and len(names) == 6
    for n in names:
        assert hasattr(lib, n)


def steps(*rows):
    return (ctypes.c_float * (3 * len(rows)))(*[v for r in rows for v in r]), len(rows)


def orth(lib, x=X, xt=0, xld=100, xs=5000, out=OUT, ot=0, old=100, os_=5000, rows=50, cols=100, count=3,
         coef=steps(*[QUINTIC] * 5), eps=1e-7, products=0, ws=WS, wsb=A):
    return lib.sl_orthogonalize(x, xt, xld, xs, out, ot, old, os_, rows, cols, count, coef[0], coef[1], eps, products, ws,
                                wsb, None)


def test_orthogonalize_argument_checks(lib):
    """Every call here is refused, or has nothing to do."""
    for kw in (dict(rows=0), dict(cols=0), dict(count=0)):
        assert orth(lib, **kw) == SL_OK
    for kw in (dict(rows=-1), dict(cols=-5), dict(count=-1), dict(rows=(1 << 20) + 1), dict(cols=1 << 40),
               dict(count=65536), dict(xld=99), dict(old=99), dict(os_=4999), dict(xs=-1),
               dict(rows=1 << 20, cols=1 << 20, xld=1 << 20, old=1 << 20, count=2, os_=1 << 40),
               dict(xld=1 << 50), dict(xs=1 << 60)):
        assert orth(lib, **kw) == SL_ERR_SHAPE, kw
    for kw in (dict(x=None), dict(out=None), dict(ws=None), dict(wsb=100), dict(xt=3), dict(ot=-1), dict(products=2),
               dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(out=X), dict(out=X + 4 * 100), dict(ws=X + 256),
               dict(ws=OUT), dict(out=WS + 256), dict(coef=(None, 5)), dict(coef=steps()),
               dict(coef=steps(*[(1.5, -0.5, 0.0)] * 17)), dict(coef=steps((nan, 0, 0))),
               dict(coef=steps((1.0, inf, 0))), dict(coef=steps((4.0, 0.0, 0.0), QUINTIC)),
               dict(coef=steps((1.0, -40.0, 0.0))), dict(coef=steps((1.0, 0.0, 31.0))), dict(coef=steps((2e4, 0.0, 0.0)))):
        assert orth(lib, **kw) == SL_ERR_INVALID_ARG, kw
    for kw in (dict(x=X + 2), dict(out=OUT + 1), dict(xt=1, x=X + 1), dict(ws=WS + 128)):
        assert orth(lib, **kw) == SL_ERR_ALIGN, kw


def muon(lib, theta=X, tt=0, m=M, grad=OUT, gt=0, rows=50, cols=100, count=3, gs=1.0, decay=0.9, lr=0.1, wd=0.0, us=1.0,
         coef=steps(QUINTIC), eps=0.0, products=1, ws=WS, wsb=A):
    return lib.sl_muon_step(theta, tt, m, grad, gt, rows, cols, count, gs, decay, 1, lr, wd, us, coef[0], coef[1], eps,
                            products, ws, wsb, None)


def test_muon_step_argument_checks(lib):
    for kw in (dict(rows=0), dict(cols=0), dict(count=0)):
        assert muon(lib, **kw) == SL_OK
    for kw in (dict(rows=-1), dict(cols=(1 << 20) + 1), dict(count=1 << 17)):
        assert muon(lib, **kw) == SL_ERR_SHAPE, kw
    for kw in (dict(theta=None), dict(m=None), dict(grad=None), dict(ws=None), dict(wsb=0), dict(tt=2), dict(gt=2),
               dict(gs=nan), dict(decay=inf), dict(lr=nan), dict(wd=inf), dict(us=-inf), dict(eps=-1.0),
               dict(lr=3e38, us=3e38), dict(lr=3e38, wd=3e38), dict(m=X), dict(grad=X + 16), dict(grad=M + 16),
               dict(ws=M + 256), dict(coef=(None, 1)), dict(products=-1)):
        assert muon(lib, **kw) == SL_ERR_INVALID_ARG, kw
    for kw in (dict(theta=X + 8), dict(m=M + 4), dict(grad=OUT + 2), dict(ws=WS + 16)):
        assert muon(lib, **kw) == SL_ERR_ALIGN, kw


def score(lib, x=X, t=0, ld=30000, targets=T, rows=8, vocab=30000, n_top=4, lp=LP, en=EN, tl=TL, ti=TI, ws=WS, wsb=A):
    return lib.sl_token_logprobs(x, t, ld, targets, rows, vocab, n_top, lp, en, tl, ti, ws, wsb, None)


def test_token_logprobs_argument_checks(lib):
    assert score(lib, rows=0) == SL_OK
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(vocab=0), dict(vocab=(1 << 22) + 1), dict(ld=29999),
               dict(ld=1 << 60)):
        assert score(lib, **kw) == SL_ERR_SHAPE, kw
    for kw in (dict(t=3), dict(n_top=-1), dict(n_top=33), dict(x=None), dict(targets=None), dict(tl=None), dict(ti=None),
               dict(ws=None), dict(wsb=1), dict(lp=X + 40), dict(en=LP + 4), dict(tl=EN), dict(ti=T), dict(ws=X),
               dict(lp=WS + 4)):
        assert score(lib, **kw) == SL_ERR_INVALID_ARG, kw
    for kw in (dict(x=X + 2), dict(t=1, x=X + 1), dict(targets=T + 4), dict(lp=LP + 2), dict(en=EN + 1), dict(tl=TL + 2),
               dict(ti=TI + 3), dict(ws=WS + 8)):
        assert score(lib, **kw) == SL_ERR_ALIGN, kw


def test_workspace_sizes(lib):
    for f in (lib.sl_orthogonalize_workspace, lib.sl_muon_step_workspace):
        assert f(0, 5, 1, 0) == f(5, 0, 1, 1) == f(5, 5, 0, 0) == 0
        assert f(-1, 5, 1, 0) == f(5, 5, 1, 2) == f(5, 1 << 21, 1, 0) == f(1 << 20, 1 << 20, 2, 0) == -1
        one, split = f(8192, 28672, 1, 0), f(8192, 28672, 1, 1)
        # three copies of X and two square matrices, twice for split operands; little else
        operands = 2 * (3 * 8192 * 28672 + 2 * 8192 * 8192)
        assert operands <= one <= 1.1 * operands
        # the weight update keeps three more square matrices at this shape
        more = 3 * 4 * 8192 * 8192 if f is lib.sl_muon_step_workspace else 0
        assert 2 * operands + more <= split <= 2.2 * operands + more
        assert f(28672, 8192, 1, 0) == one and 3 * one // 4 < f(8192, 28672, 4, 0) // 4 <= one + 4096
    f = lib.sl_token_logprobs_workspace
    assert f(0, 10, 0, 0) == 0 and f(4, 0, 0, 0) == f(4, 10, 7, 0) == f(4, 10, 0, 33) == f(-1, 10, 0, 0) == -1
    assert 0 < f(1, 262208, 1, 0) <= f(1, 262208, 1, 20) < 1 << 16
    assert f(4096, 262208, 1, 5) < 1 << 23


def test_binding_refusals():
    """Host tensors and mismatched arguments raise before the library is called."""
    import communication_efficient_distributed_amd as sl
    x = torch.zeros(4, 6)
    with pytest.raises(ValueError):
        sl.orthogonalize(x)
    with pytest.raises(ValueError):
        sl.muon_step(x, x.clone(), x.clone(), lr=0.1)
    with pytest.raises(ValueError):
        sl.token_logprobs(x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        sl.orthogonalize([1.0])
    with pytest.raises(ValueError):
        sl.orthogonalize_workspace(4, 4, 1, "bf16")


C_CALLER = r"""
#include <stddef.h>
#include <stdio.h>
#include "sparseloco_ops.h"

int main(void) {
    const float steps[3] = {1.5f, -0.5f, 0.0f};
    float* fake = (float*)(unsigned long)0x10000;        /* never dereferenced */
    int bad = 0;
    bad |= sl_orthogonalize(fake, SL_F32, 4, 0, fake, SL_F32, 4, 0, 4, 4, 1, steps, 1, 0.0f, SL_PRODUCTS_F16, NULL, 0,
                            NULL) != SL_ERR_INVALID_ARG;
    bad |= sl_muon_step(fake, SL_F32, fake, fake, SL_F32, 0, 4, 1, 1.0f, 0.9f, 1, 0.1f, 0.0f, 1.0f, steps, 1, 0.0f,
                        SL_PRODUCTS_SPLIT, NULL, 0, NULL) != SL_OK;
    bad |= sl_token_logprobs(fake, SL_BF16, 3, NULL, 1, 4, 0, NULL, NULL, NULL, NULL, NULL, 0, NULL) != SL_ERR_SHAPE;
    bad |= sl_orthogonalize_workspace(4, 4, 1, SL_PRODUCTS_SPLIT) <= 0;
    puts(bad ? "FAIL" : "OK");
    return bad;
}
"""


def test_header_compiles_as_c99_and_links(lib, tmp_path):
    src, exe = tmp_path / "caller.c", tmp_path / "caller"
    src.write_text(C_CALLER)
    libdir = os.path.dirname(lib._name)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    str(src), "-L", libdir, "-lsparseloco", f"-Wl,-rpath,{libdir}", "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.split() == ["OK"], (out.stdout, out.stderr)


@pytest.mark.parametrize("source", ["newton.hip", "newton_narrow.hip", "logprobs.hip"])
def test_no_scratch_and_no_spills(source, tmp_path):
    spec = importlib.util.spec_from_file_location("resources", os.path.join(ROOT, "tests", "test_kernel_resources.py"))
    resources = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(resources)
    kernels = resources._resources(source, tmp_path)
    assert kernels, "the compiler printed no resource remarks"
    for k in kernels:
        for what in ("ScratchSize [bytes/lane]", "VGPRs Spill"):
            assert k.get(what, 0) == 0, (k["name"], k)
        # scalar registers go to vector lanes: a few of this kernel's arguments do
        assert k.get("SGPRs Spill", 0) <= (6 if "narrow_apply_kernel" in k["name"] else 0), (k["name"], k)
