"""AdamW over many tensors at once: the norm of all gradients with the factor that
clips them, the AdamW step with its moments in 32 bits, and the step with its
moments in 8 bits (ma_grad_norm, ma_adamw_many_step, ma_adamw8_many_step and
ma_adamw8_many_values of include/microadam.h; the formulas stand there).

Every call takes a whole list of tensors where they lie, of fp32 and bf16 in any
mixture.  The moments of a list are flat arrays of state_size(params) elements:
tensor i has its own at starts(params)[i], in the order in which its elements lie
in memory, and what lies between is not used.  A parameter is dense (contiguous, or
a permutation of that, as a transposed or channels-last one is), and its gradient
lies like it.  A gradient of None leaves its parameter and that one's moments
alone.

Calls are asynchronous on `stream` (default: the current stream of the tensors'
device), allocate workspace and results through torch on that stream and can be
captured into a graph; a graph that is replayed as a training step takes the
step's number `t`, and `lr` where it changes, as tensors, which are read at every
replay.  A tensor that another stream made must be ordered before `stream` by the
caller, as for any kernel, and kept until its work there is done
(Tensor.record_stream).  Bits repeat from call to call.
"""
from __future__ import annotations

import ctypes as C
import math

from . import _lib as _L
from .muon import _place, _workspace, changed

BLOCK = 256   # elements of a tensor that share the scales of their 8-bit moments


def starts(params) -> list[int]:
    """Where each tensor's moments begin in a list's state arrays."""
    out, at = [], 0
    for p in params:
        out.append(at)
        at += -(-p.numel() // BLOCK) * BLOCK
    return out


def state_size(params) -> int:
    """Elements of a list's state arrays (a multiple of 256)."""
    return sum(-(-p.numel() // BLOCK) * BLOCK for p in params)


def views(state, params) -> list:
    """The part of a state array that belongs to each tensor, in the tensor's shape."""
    return [state[a:a + p.numel()].as_strided(p.shape, p.stride(), state.storage_offset() + a)
            for p, a in zip(params, starts(params))]


def _dense(t) -> bool:
    """Whether its elements fill a stretch of memory, in whatever order."""
    if t.is_contiguous():
        return True
    step = 1
    for s, n in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1):
        if s != step:
            return False
        step *= n
    return True


def _like(g, p) -> bool:
    """Whether gradient and parameter have the same elements in the same places."""
    if g.shape != p.shape:
        return False
    if g.is_contiguous() and p.is_contiguous():
        return True
    return g.numel() < 2 or (_dense(g) and all(a == b for a, b, n in zip(g.stride(), p.stride(), p.shape) if n > 1))


def _type(t, what: str) -> int:
    import torch
    _L.require(t.dtype in (torch.float32, torch.bfloat16), f"{what} must be fp32 or bf16")
    return _L.MA_TYPE_F32 if t.dtype == torch.float32 else _L.MA_TYPE_BF16


def _list(params, grads):
    """The ma_tensor array of a list, its length, its device and the states' size."""
    _L.require(len(params) == len(grads), "there must be a gradient, or None, for every parameter")
    rows = (_L.Tensor * len(params))()
    device, count, at = None, 0, 0
    for p, g in zip(params, grads):
        n = p.numel()
        if device is None:
            device = p.device
            _L.require(p.is_cuda, "parameters must be CUDA tensors")
        if g is not None:
            _L.require(p.device == device and g.device == device, "parameters and gradients must be on one device")
            _L.require(_dense(p), "parameters must be dense")
            _L.require(_like(g, p), "a gradient must have its parameter's shape and strides")
            r = rows[count]
            r.param, r.grad, r.n, r.at = p.data_ptr(), g.data_ptr(), n, at
            r.p_type, r.g_type = _type(p, "parameters"), _type(g, "gradients")
            count += 1
        at += -(-n // BLOCK) * BLOCK
    return rows, count, device, at


def _state(t, what: str, dtypes, size: int, device):
    _L.require(t.dtype in dtypes and t.is_contiguous() and t.numel() == size and t.device == device,
               f"{what} must be contiguous {dtypes[0]} of {size} elements on the parameters' device")


def _one(t, what: str, dtype, device):
    _L.require(t.dtype == dtype and t.numel() == 1 and t.device == device,
               f"{what} must be one {dtype} on the parameters' device")
    return t.data_ptr()


def _arguments(t, lr, beta1, beta2, eps, wd, scale, device):
    import torch
    a = _L.AdamwArgs(0.0, beta1, beta2, eps, wd, 0, None, None, None)
    if torch.is_tensor(t):
        a.t_dev = _one(t, "t", torch.int64, device)
    else:
        a.t = int(t)
    if torch.is_tensor(lr):
        a.lr_dev = _one(lr, "lr", torch.float32, device)
    else:
        a.lr = lr
    if scale is not None:
        a.scale = _one(scale, "scale", torch.float32, device)
    return a


def grad_norm(grads, max_norm: float = math.inf, t=None, out=None, stream=None):
    """(norm, scale), two fp32 tensors of one element on the GPU: the norm of all
    gradients (None is passed over), and the factor min(1, max_norm / (norm + 1e-6))
    that clips them, for the steps' `scale`.  Where the norm is not finite the
    factor is NaN, and a step with it changes nothing.  t: an int64 tensor, a
    count of steps that is raised by one if the norm is finite.  out: fp32 of two
    elements for both."""
    import torch
    grads = [g for g in grads if g is not None]
    _L.require(len(grads) > 0 or out is not None, "there must be a gradient, or out")
    device = out.device if out is not None else grads[0].device
    _L.require(device.type == "cuda", "gradients must be CUDA tensors")
    rows = (_L.Tensor * len(grads))()
    for r, g in zip(rows, grads):
        _L.require(g.device == device, "gradients must be on one device")
        _L.require(_dense(g), "gradients must be dense")
        r.grad, r.n, r.g_type = g.data_ptr(), g.numel(), _type(g, "gradients")
    L = _L.lib()
    nbytes = L.ma_grad_norm_workspace(len(grads))
    s, place = _place(device, stream)
    with place:
        if out is None:
            out = torch.empty(2, dtype=torch.float32, device=device)
        _state(out, "out", (torch.float32,), 2, device)
        ws = _workspace(nbytes, device)
        _L.check(L.ma_grad_norm(len(grads), rows, max_norm, out.data_ptr(), None if t is None else _one(t, "t", torch.int64, device),
                                ws.data_ptr(), nbytes, s.cuda_stream))
    changed(out, *(() if t is None else (t,)))
    return out.unbind()


def adamw_step(params, grads, m, v, t, lr=1e-3, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, wd: float = 0.0,
               scale=None, master=None, stream=None):
    """One AdamW step, in place on params, m and v: with x = scale grads, m <-
    beta1 m + (1 - beta1) x; v <- beta2 v + (1 - beta2) x^2; p <- p - lr (m^ / (sqrt(v^)
    + eps) + wd p) with m^ = m / (1 - beta1^t), v^ = v / (1 - beta2^t).  m, v: fp32
    of state_size(params) elements, zeros before the first step.  t: this step's
    number from 1, an int or an int64 tensor on the GPU (below 1 there: nothing
    changes); lr: a float or an fp32 tensor.  scale: an fp32 tensor, the gradients'
    factor (grad_norm's); NaN: nothing changes.  master: fp32 like m, the 32-bit
    copies of the bf16 parameters, which take the step in their place and are
    rounded into them."""
    import torch
    rows, count, device, size = _list(params, grads)
    if not count:
        return
    f32 = (torch.float32,)
    _state(m, "m", f32, size, device)
    _state(v, "v", f32, size, device)
    if master is not None:
        _state(master, "master", f32, size, device)
    a = _arguments(t, lr, beta1, beta2, eps, wd, scale, device)
    s, place = _place(device, stream)
    with place:
        _L.check(_L.lib().ma_adamw_many_step(count, rows, C.byref(a), None if master is None else master.data_ptr(), m.data_ptr(),
                                             v.data_ptr(), size, s.cuda_stream))
    changed(m, v, *(() if master is None else (master,)), *(p for p, g in zip(params, grads) if g is not None))


def _moments8(cm, cv, sm, sr, size, device):
    import torch
    _state(cm, "cm", (torch.int8,), size, device)
    _state(cv, "cv", (torch.uint8,), size, device)
    _state(sm, "sm", (torch.float32,), size // BLOCK, device)
    _state(sr, "sr", (torch.float32,), size // BLOCK, device)
    return cm.data_ptr(), cv.data_ptr(), sm.data_ptr(), sr.data_ptr()


def adamw8_step(params, grads, cm, cv, sm, sr, t, lr=1e-3, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                wd: float = 0.0, scale=None, master=None, stream=None):
    """adamw_step with the moments in 8 bits: cm int8 and cv uint8 codes of
    state_size(params) elements, sm and sr fp32 scales of one for 256 of them,
    updated in place, all zeros before the first step."""
    import torch
    rows, count, device, size = _list(params, grads)
    if not count:
        return
    state = _moments8(cm, cv, sm, sr, size, device)
    if master is not None:
        _state(master, "master", (torch.float32,), size, device)
    a = _arguments(t, lr, beta1, beta2, eps, wd, scale, device)
    s, place = _place(device, stream)
    with place:
        _L.check(_L.lib().ma_adamw8_many_step(count, rows, C.byref(a), None if master is None else master.data_ptr(), *state, size,
                                              s.cuda_stream))
    changed(cm, cv, sm, sr, *(() if master is None else (master,)), *(p for p, g in zip(params, grads) if g is not None))


def adamw8_values(cm, cv, sm, sr, stream=None):
    """(m, v), the fp32 moments that an 8-bit state stands for."""
    import torch
    size, device = cm.numel(), cm.device
    _L.require(cm.is_cuda, "cm must be a CUDA tensor")
    _L.require(size % BLOCK == 0, f"cm must have a multiple of {BLOCK} elements")
    state = _moments8(cm, cv, sm, sr, size, device)
    s, place = _place(device, stream)
    with place:
        m, v = (torch.empty(size, dtype=torch.float32, device=device) for _ in range(2))
        _L.check(_L.lib().ma_adamw8_many_values(size, *state, m.data_ptr(), v.data_ptr(), s.cuda_stream))
    return m, v
