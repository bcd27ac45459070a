"""The Muon operators: orthogonalizing an update by Newton-Schulz products, the
Muon step, and the Muon step whose momentum is held in 8 bits.

Muon is for the matrices of a model; MicroAdam takes the rest.  Every call works
on one matrix [rows, cols] or on a batch of equally shaped ones [..., rows,
cols] in one go (ma_orthogonalize, ma_muon_step, ma_muon8_step and
ma_momentum8_values of include/microadam.h; the formulas and their rounding
stand there).  Calls are asynchronous on `stream` (default: the current stream
of the tensors' device), allocate their workspace and new results through torch
on that stream and can be captured into a graph.  A tensor that another stream
made must be ordered before `stream` by the caller, as for any kernel, and kept
until its work there is done (Tensor.record_stream), and so must what another
stream does with a result.

Products are rounded to 11 bits: a result is off by about 2e-3 for random
matrices, by more where singular values are far apart (the header gives
figures).  The same call on the same sizes repeats its bits; a matrix alone and
the same matrix in a larger batch can differ by roundings.  `coefficients`
that could carry a singular value past 1.95 or an eigenvalue of a I + b A + c A A
past 15 are refused (MicroAdamError): the products' number format ends there.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import functools
import math

from . import _lib as _L

# five steps with these bring singular values from about 0.01..1 into 0.68..1.2
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
BLOCK = 256   # elements of a row that share one scale of the 8-bit momentum


def rms_scale(rows: int, cols: int) -> float:
    """0.2 sqrt(max(rows, cols)): with this `scale` an update's entries have a
    root mean square of about 0.2 lr, like AdamW's, so that one learning rate
    serves both."""
    return 0.2 * math.sqrt(max(rows, cols))


@functools.lru_cache(maxsize=64)
def _host_coefficients(coefficients, steps: int):
    """The C array of (a, b, c) for every step: `coefficients` is one triple or
    `steps` of them."""
    _L.require(steps >= 1, "steps must be at least 1")
    rows = (coefficients,) * steps if not any(isinstance(v, tuple) for v in coefficients) else coefficients
    _L.require(len(rows) == steps and all(isinstance(r, tuple) and len(r) == 3 for r in rows),
               "coefficients must be one triple (a, b, c) or one for each step")
    return (C.c_float * (3 * steps))(*(v for r in rows for v in r))


def _coefficients(coefficients, steps: int):
    if type(coefficients) is not tuple or not all(type(v) is float for v in coefficients):
        # any sequences of numbers; as tuples of floats they are told apart by value
        coefficients = tuple(tuple(map(float, r)) if hasattr(r, "__len__") and getattr(r, "ndim", 1) else float(r)
                             for r in coefficients)
    return _host_coefficients(coefficients, int(steps))


def _batched(t, what: str):
    """(batch, rows, cols, row stride, batch stride) of a [..., rows, cols] tensor."""
    _L.require(t.is_cuda and t.dim() >= 2, f"{what} must be a CUDA tensor of at least two dimensions")
    rows, cols = t.shape[-2:]
    sr, sc = t.stride()[-2:]
    _L.require(sc == 1 or cols <= 1, f"{what}'s last dimension must be contiguous")
    batch, sb = 1, 0
    for n, s in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
        if n == 1:
            continue
        _L.require(batch <= 1 or s == sb * batch, f"{what}'s leading dimensions must have one stride")
        batch, sb = batch * n, (s if batch == 1 else sb)
    return batch, rows, cols, sr, sb


def _type(t, what: str) -> int:
    import torch
    _L.require(t.dtype in (torch.float32, torch.bfloat16), f"{what} must be fp32 or bf16")
    return _L.MA_TYPE_F32 if t.dtype == torch.float32 else _L.MA_TYPE_BF16


def _place(device, stream):
    """The stream to use, and a context for allocations and the call: in it torch
    allocates on that stream, and its device is the current one (a device's
    default stream has no other mark)."""
    import torch
    current = torch.cuda.current_stream(device)
    s = current if stream is None else stream
    _L.require(s.device == device, "the stream must be of the tensors' device")
    if s == current and torch.cuda.current_device() == device.index:
        return s, contextlib.nullcontext()
    return s, torch.cuda.stream(s)


def _workspace(nbytes: int, device):
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def changed(*tensors) -> None:
    """Tells autograd that a call has written them in place, so that a backward
    pass that needs what they held before raises."""
    import torch
    torch.autograd.graph.increment_version(tensors)


def orthogonalize(x, steps: int = 5, coefficients=COEFFICIENTS, eps: float = 1e-7, out=None, stream=None):
    """x [..., rows, cols] (fp32 or bf16) orthogonalized, as bf16: X = x /
    max(|x|_F, eps), then `steps` times X <- (a I + b A + c A A) X with A = X X^T
    on the shorter side.  out: a bf16 tensor of x's shape (x itself if it is
    bf16); by default a new one.  The result carries no gradient."""
    import torch
    batch, rows, cols, sr, sb = _batched(x, "x")
    kind = _type(x, "x")
    k = _coefficients(coefficients, steps)
    L = _L.lib()
    nbytes = L.ma_orthogonalize_workspace(batch, rows, cols)
    s, place = _place(x.device, stream)
    with place:
        if out is None:
            out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
        _L.require(out.device == x.device and out.shape == x.shape and out.dtype == torch.bfloat16,
                   "out must be a bf16 tensor of x's shape and device")
        _, _, _, osr, osb = _batched(out, "out")
        ws = _workspace(nbytes, x.device)
        _L.check(L.ma_orthogonalize(batch, rows, cols, x.data_ptr(), kind, sr, sb, out.data_ptr(), osr, osb, steps, k, eps,
                                    ws.data_ptr(), nbytes, s.cuda_stream))
    changed(out)
    return out


def _step_arguments(params, grads, lr, wd, beta, scale):
    import torch
    batch, rows, cols, psr, psb = _batched(params, "params")
    kind = _type(params, "params")
    _L.require(grads.dtype in (torch.bfloat16, torch.int16) and grads.shape == params.shape
               and grads.device == params.device, "grads must be bf16 (or int16 bits) of params' shape and device")
    _, _, _, gsr, gsb = _batched(grads, "grads")
    if scale is None:
        scale = rms_scale(rows, cols)
    return batch, rows, cols, (params.data_ptr(), kind, psr, psb, grads.data_ptr(), gsr, gsb), (lr, beta, wd, scale)


def muon_step(params, grads, momentum, lr: float = 1e-3, beta: float = 0.95, wd: float = 0.0, nesterov: bool = True,
              scale: float | None = None, steps: int = 5, coefficients=COEFFICIENTS, eps: float = 1e-7, stream=None):
    """One Muon step, in place on params (fp32 or bf16) and momentum (fp32,
    contiguous, zeros before the first step): momentum <- beta momentum +
    (1 - beta) grads; U = beta momentum + (1 - beta) grads (nesterov) or the
    momentum; params <- params (1 - lr wd) - lr scale orthogonalize(U).  grads:
    bf16 (or int16 bits).  scale: default rms_scale(rows, cols)."""
    import torch
    batch, rows, cols, arrays, hyper = _step_arguments(params, grads, lr, wd, beta, scale)
    _L.require(momentum.dtype == torch.float32 and momentum.shape == params.shape and momentum.is_contiguous()
               and momentum.device == params.device, "momentum must be contiguous fp32 of params' shape and device")
    k = _coefficients(coefficients, steps)
    L = _L.lib()
    nbytes = L.ma_orthogonalize_workspace(batch, rows, cols)
    s, place = _place(params.device, stream)
    with place:
        ws = _workspace(nbytes, params.device)
        _L.check(L.ma_muon_step(batch, rows, cols, *arrays, momentum.data_ptr(), *hyper, int(nesterov), steps, k, eps,
                                ws.data_ptr(), nbytes, s.cuda_stream))
    changed(params, momentum)


def scales_shape(shape):
    """Shape of the 8-bit momentum's scales for parameters of this shape."""
    return (*shape[:-1], -(-shape[-1] // BLOCK))


def _require_momentum8(codes, scales, device):
    import torch
    _L.require(codes.dtype == torch.int8 and codes.is_contiguous() and codes.device == device,
               "codes must be contiguous int8 on the parameters' device")
    _L.require(scales.dtype == torch.float32 and scales.is_contiguous() and scales.device == device
               and tuple(scales.shape) == scales_shape(codes.shape),
               f"scales must be contiguous fp32, one for each {BLOCK} elements of a row")


def muon8_step(params, grads, codes, scales, lr: float = 1e-3, beta: float = 0.95, wd: float = 0.0,
               nesterov: bool = True, scale: float | None = None, steps: int = 5, coefficients=COEFFICIENTS,
               eps: float = 1e-7, stream=None):
    """muon_step with the momentum in 8 bits: codes (int8, params' shape) and
    scales (fp32, scales_shape(params.shape)), contiguous, updated in place,
    zeros before the first step."""
    batch, rows, cols, arrays, hyper = _step_arguments(params, grads, lr, wd, beta, scale)
    _L.require(codes.shape == params.shape, "codes must have params' shape")
    _require_momentum8(codes, scales, params.device)
    k = _coefficients(coefficients, steps)
    L = _L.lib()
    nbytes = L.ma_orthogonalize_workspace(batch, rows, cols)
    s, place = _place(params.device, stream)
    with place:
        ws = _workspace(nbytes, params.device)
        _L.check(L.ma_muon8_step(batch, rows, cols, *arrays, codes.data_ptr(), scales.data_ptr(), *hyper, int(nesterov),
                                 steps, k, eps, ws.data_ptr(), nbytes, s.cuda_stream))
    changed(params, codes, scales)


def momentum8_values(codes, scales, out=None, stream=None):
    """The fp32 values that an 8-bit momentum stands for (code times scale)."""
    import torch
    _L.require(codes.is_cuda and codes.dim() >= 1, "codes must be a CUDA tensor")
    _require_momentum8(codes, scales, codes.device)
    s, place = _place(codes.device, stream)
    with place:
        if out is None:
            out = torch.empty(codes.shape, dtype=torch.float32, device=codes.device)
        _L.require(out.dtype == torch.float32 and out.shape == codes.shape and out.is_contiguous()
                   and out.device == codes.device, "out must be contiguous fp32 of codes' shape and device")
        cols = codes.shape[-1]
        _L.check(_L.lib().ma_momentum8_values(codes.numel() // cols if cols else 0, cols, codes.data_ptr(),
                                              scales.data_ptr(), out.data_ptr(), s.cuda_stream))
    changed(out)
    return out
