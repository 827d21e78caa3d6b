"""Binding of the operators declared in include/sparseloco_ops.h: the matrix
update (orthogonalisation by Newton-Schulz products, the momentum step that uses
it) and the log probabilities of given tokens.

Marshalling only, as in _lib.py: device pointers, sizes and the current HIP
stream go to the library, a non-OK status raises, and there is no fallback.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import _check, load

SL_MAX_ALTERNATIVES = 32
SL_PRODUCTS_F16 = 0
SL_PRODUCTS_SPLIT = 1
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_PRODUCTS = {"f16": SL_PRODUCTS_F16, "split": SL_PRODUCTS_SPLIT}

# (a, b, c) of each step X <- a X + (b A + c A A) X, A = X X^T: singular values
# of 0.003 and more reach [0.68, 1.21] in five steps.
SL_NEWTON_SCHULZ = ((3.4445, -4.7750, 2.0315),) * 5
_STANDARD = (ctypes.c_float * 15)(*[v for step in SL_NEWTON_SCHULZ for v in step])


def _gpu(t: torch.Tensor, name: str, dtypes) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {', '.join(str(d) for d in dtypes)} (got {t.dtype})")
    return t


def _buffer(t: torch.Tensor | None, name: str, dtype, shape, device) -> int | None:
    """Address of a contiguous GPU tensor of this type, shape and device (None stays None)."""
    if t is None:
        return None
    _gpu(t, name, (dtype,))
    if t.shape != shape:
        raise ValueError(f"{name} must be of shape {list(shape)} (got {list(t.shape)})")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# The current stream's handle without a Stream object around it, where torch has it.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(name: str, device, args, stream) -> None:
    """Calls the library with the device current and the stream last; torch's
    device guard only where another device is current, since it costs as much
    as a kernel launch."""
    handle = _current_stream(device.index) if stream is None else \
        int(stream.cuda_stream if hasattr(stream, "cuda_stream") else stream)
    fn = getattr(load(), name)
    if torch.cuda.current_device() == device.index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            status = fn(*args, handle)
    if status:
        _check(name, status)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """New memory for a call on `stream` (None: the current one). It is that
    stream's own: memory of the current one may still be in use by work queued
    there, which `stream` does not wait for."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _strided(t: torch.Tensor, name: str):
    """(rows, cols, count, row stride, matrix stride) of a [rows, cols] or
    [count, rows, cols] tensor whose columns are adjacent."""
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be [rows, cols] or [count, rows, cols]")
    rows, cols = t.shape[-2:]
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have adjacent columns (stride 1)")
    ld = t.stride(-2) if rows > 1 else max(cols, 1)
    if rows > 1 and ld < cols:
        raise ValueError(f"{name}'s rows must not overlap")
    count = t.shape[0] if t.dim() == 3 else 1
    return rows, cols, count, ld, t.stride(0) if t.dim() == 3 and count > 1 else 0


def _coefficients(steps):
    if steps is SL_NEWTON_SCHULZ:
        return _STANDARD, len(steps)
    flat = [float(v) for step in steps for v in step]
    if len(flat) != 3 * len(steps):
        raise ValueError("coefficients must be (a, b, c) for each step")
    return (ctypes.c_float * max(len(flat), 1))(*flat), len(steps)


def _products(products, dtype) -> int:
    if products is None:
        return SL_PRODUCTS_SPLIT if dtype == torch.float32 else SL_PRODUCTS_F16
    if products not in _PRODUCTS:
        raise ValueError("products must be None, 'f16' or 'split'")
    return _PRODUCTS[products]


def _workspace(fn: str, need: int, workspace, device, stream):
    """(workspace, address, bytes): the caller's, checked, or one from torch's
    allocator; the first is held until the call is made."""
    if need < 0:
        raise ValueError(f"{fn}: sizes outside the documented range")
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = _empty(need, torch.uint8, device, stream)
        return workspace, workspace.data_ptr(), need
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise ValueError(f"{fn}: workspace of {have} bytes, {need} needed")
    if not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"{fn}: workspace must be contiguous and on {device}")
    return workspace, workspace.data_ptr(), have


def orthogonalize_workspace(rows: int, cols: int, count: int = 1, products: str = "f16") -> int:
    """Bytes of workspace that sl_orthogonalize needs for matrices of this size."""
    return load().sl_orthogonalize_workspace(rows, cols, count, _products(products, None))


def muon_step_workspace(rows: int, cols: int, count: int = 1, products: str = "f16") -> int:
    """Bytes of workspace that sl_muon_step needs for matrices of this size."""
    return load().sl_muon_step_workspace(rows, cols, count, _products(products, None))


def token_logprobs_workspace(rows: int, vocab: int, dtype: torch.dtype, n_top: int = 0) -> int:
    """Bytes of workspace that sl_token_logprobs needs."""
    return load().sl_token_logprobs_workspace(rows, vocab, _TYPES[dtype], n_top)


def sl_orthogonalize(x: torch.Tensor, out: torch.Tensor, coefficients=SL_NEWTON_SCHULZ, eps: float = 1e-7,
                     products: str | None = None, workspace: torch.Tensor | None = None, stream=None) -> None:
    """out = the Newton-Schulz orthogonalisation of x ([rows, cols] or [count,
    rows, cols], float32, bfloat16 or float16, adjacent columns; rows and
    matrices may be strided).  products: 'f16' (within about 1e-3 of the exact
    result) or 'split' (as fp32 arithmetic, three times the products); by default
    'split' for a float32 out and 'f16' for a 16-bit one.  workspace: a buffer
    of orthogonalize_workspace() bytes to use again; by default one from torch's
    allocator."""
    _gpu(x, "x", _TYPES), _gpu(out, "out", _TYPES)
    if out.device != x.device:
        raise ValueError(f"out must be on {x.device} (got {out.device})")
    if x.shape != out.shape:
        raise ValueError("x and out shapes differ")
    rows, cols, count, x_ld, x_stride = _strided(x, "x")
    *_, out_ld, out_stride = _strided(out, "out")
    mode = _products(products, out.dtype)
    steps, n_steps = _coefficients(coefficients)
    need = load().sl_orthogonalize_workspace(rows, cols, count, mode)
    keep, ws, ws_bytes = _workspace("sl_orthogonalize", need, workspace, x.device, stream)
    _call("sl_orthogonalize", x.device,
          (x.data_ptr(), _TYPES[x.dtype], x_ld, x_stride, out.data_ptr(), _TYPES[out.dtype], out_ld, out_stride,
           rows, cols, count, steps, n_steps, eps, mode, ws, ws_bytes), stream)


def sl_muon_step(theta: torch.Tensor, momentum: torch.Tensor, grad: torch.Tensor, lr: float, grad_scale: float = 1.0,
                 decay: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0, update_scale: float = 1.0,
                 coefficients=SL_NEWTON_SCHULZ, eps: float = 1e-7, products: str | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> None:
    """One weight update of theta ([rows, cols] or [count, rows, cols], float32
    or bfloat16) in place: g = grad_scale * grad, momentum <- decay * momentum +
    g (float32, in place), u = g + decay * momentum (nesterov) or momentum,
    theta <- theta * (1 - lr * weight_decay) - lr * update_scale *
    orthogonalize(u).  As an outer update, grad is the sum of sl_aggregate and
    grad_scale 1 / n_peers.  products and workspace as for sl_orthogonalize
    (default by theta's type; 'split' is within about 1e-5 for large matrices
    that are not square), the latter of muon_step_workspace() bytes."""
    _gpu(theta, "theta", (torch.float32, torch.bfloat16)), _gpu(grad, "grad", (torch.float32, torch.bfloat16))
    if theta.dim() not in (2, 3):
        raise ValueError("theta must be [rows, cols] or [count, rows, cols]")
    dev, shape = theta.device, theta.shape
    buffers = (_buffer(theta, "theta", theta.dtype, shape, dev), _TYPES[theta.dtype],
               _buffer(momentum, "momentum", torch.float32, shape, dev),
               _buffer(grad, "grad", grad.dtype, shape, dev), _TYPES[grad.dtype])
    rows, cols = shape[-2:]
    count = shape[0] if len(shape) == 3 else 1
    mode = _products(products, theta.dtype)
    steps, n_steps = _coefficients(coefficients)
    need = load().sl_muon_step_workspace(rows, cols, count, mode)
    keep, ws, ws_bytes = _workspace("sl_muon_step", need, workspace, dev, stream)
    _call("sl_muon_step", dev,
          (*buffers, rows, cols, count, grad_scale, decay, int(bool(nesterov)), lr, weight_decay, update_scale,
           steps, n_steps, eps, mode, ws, ws_bytes), stream)


def sl_token_logprobs(logits: torch.Tensor, targets: torch.Tensor | None, logprob: torch.Tensor | None,
                      entropy: torch.Tensor | None, top_logprob: torch.Tensor | None = None,
                      top_index: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      stream=None) -> None:
    """For each row of logits ([rows, vocab], float32, bfloat16 or float16, rows
    may be strided): logprob [rows] = log p(targets[row]) (0 where the target is
    outside the vocabulary), entropy [rows], and the likeliest tokens
    top_index [rows, n_top] (int32, ties to the lower token, -1 where none is
    left) with their top_logprob.  Any output but not its partner may be None."""
    _gpu(logits, "logits", _TYPES)
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab, _, ld, _ = _strided(logits, "logits")
    if vocab == 0:
        raise ValueError("logits must have a vocabulary")
    if (top_logprob is None) != (top_index is None):
        raise ValueError("top_logprob and top_index come together")
    if logprob is not None and targets is None:
        raise ValueError("logprob needs targets")
    n_top = 0 if top_index is None else top_index.shape[-1]
    dev, kind = logits.device, _TYPES[logits.dtype]
    buffers = (_buffer(logprob, "logprob", torch.float32, (rows,), dev),
               _buffer(entropy, "entropy", torch.float32, (rows,), dev),
               _buffer(top_logprob, "top_logprob", torch.float32, (rows, n_top), dev),
               _buffer(top_index, "top_index", torch.int32, (rows, n_top), dev))
    target = _buffer(targets, "targets", torch.int64, (rows,), dev)
    need = load().sl_token_logprobs_workspace(rows, vocab, kind, n_top)
    keep, ws, ws_bytes = _workspace("sl_token_logprobs", need, workspace, dev, stream)
    _call("sl_token_logprobs", dev,
          (logits.data_ptr(), kind, ld, target, rows, vocab, n_top, *buffers, ws, ws_bytes), stream)


# Convenience wrappers that allocate outputs with torch (device memory only),
# as memory of the stream they run on.

def orthogonalize(x: torch.Tensor, out_dtype: torch.dtype | None = None, coefficients=SL_NEWTON_SCHULZ,
                  eps: float = 1e-7, products: str | None = None, workspace: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """sl_orthogonalize into a new tensor of out_dtype (default x's type)."""
    _gpu(x, "x", _TYPES)
    out = _empty(x.shape, out_dtype or x.dtype, x.device, stream)
    sl_orthogonalize(x, out, coefficients, eps, products, workspace, stream)
    return out


def muon_step(theta: torch.Tensor, momentum: torch.Tensor, grad: torch.Tensor, lr: float, **kw) -> torch.Tensor:
    """sl_muon_step (theta and momentum in place); returns theta."""
    sl_muon_step(theta, momentum, grad, lr, **kw)
    return theta


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, n_top: int = 0, workspace: torch.Tensor | None = None,
                   stream=None):
    """sl_token_logprobs into new tensors: (logprob, entropy, top_logprob,
    top_index), the last two None for n_top = 0."""
    _gpu(logits, "logits", _TYPES)
    rows, dev = logits.shape[0], logits.device
    logprob, entropy = _empty((2, rows), torch.float32, dev, stream).unbind(0)
    top_logprob = _empty((rows, n_top), torch.float32, dev, stream) if n_top else None
    top_index = _empty((rows, n_top), torch.int32, dev, stream) if n_top else None
    sl_token_logprobs(logits, targets, logprob, entropy, top_logprob, top_index, workspace, stream)
    return logprob, entropy, top_logprob, top_index
