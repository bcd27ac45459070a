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

import contextlib
import ctypes as C
import functools
import math

from . import _lib as _L
from .muon import _place, _workspace

_HERE = contextlib.nullcontext()
BLOCK = 256   # elements of a tensor that share the scales of their 8-bit moments
_FLT_MIN, _FLT_MAX = 2.0 ** -126, 2.0 ** 128 - 2.0 ** 104


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
    params = _sequence(params)
    return [state[a:a + p.numel()].as_strided(p.shape, p.stride(), state.storage_offset() + a)
            for p, a in zip(params, starts(params))]


@functools.lru_cache(maxsize=None)
def _native():
    """The module that reads lists of tensors (csrc/tensors.cpp)."""
    import torch  # noqa: F401  its libraries come first
    try:
        from . import _tensors
    except ImportError as e:
        raise ImportError("_tensors.so is not built; run `python -m memory_compressed_adaptive_amd.build` "
                          "(or __graft_entry__.build())") from e
    return _tensors


@functools.lru_cache(maxsize=None)
def _device(index: int):
    import torch
    return torch.device("cuda", index)


def require_dense(params) -> None:
    """ValueError unless every parameter is one that the steps take."""
    params = _sequence(params)
    _native().rows(params, params)


def layout(params) -> bytes:
    """The types, devices, shapes and strides of all parameters, which say how their moments lie and
    whether the steps take them."""
    return _native().layout(params)


def missing(params, grads) -> int:
    """How many parameters have None for a gradient; -1 if the steps do not take some gradient
    as it is (fp32 or bf16, lying like its parameter)."""
    return _native().missing(params, grads)


def check_numbers(lr, beta1, beta2, eps, wd) -> None:
    """ValueError for numbers that the steps refuse."""
    _L.require(0.0 <= beta1 < 1.0 and 0.0 <= beta2 < 1.0, "beta1 and beta2 must be in [0, 1)")
    _L.require(_FLT_MIN <= eps <= _FLT_MAX, "eps must be positive and finite (a normal fp32)")
    _L.require(math.isfinite(lr) and 0.0 <= wd < math.inf, "lr and weight decay must be finite, weight decay not negative")


def _sequence(x):
    """A list as it is; what an iterator yields, kept until the call is made: the rows that are read
    from it hold addresses only."""
    return x if isinstance(x, (list, tuple)) else list(x)


def _state(t, what: str, dtype, size: int, device):
    at = _native().data(t, dtype, size, device)
    if at is None:
        raise ValueError(f"{what} must be contiguous {dtype} of {size} elements on the device of the tensors")
    return at


def _one(t, what: str, dtype, device):
    at = _native().data(t, dtype, 1, device)
    if at is None:
        raise ValueError(f"{what} must be one {dtype} on the device of the tensors")
    return at


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


def _stream(device, stream):
    """The handle of the stream to use, and a context for allocations and the call."""
    if stream is None:
        handle = _native().stream(device.index)
        if handle is not None:
            return handle, _HERE
    s, place = _place(device, stream)
    return s.cuda_stream, place


def grad_norm(grads, max_norm: float = math.inf, t=None, out=None, stream=None):
    """(norm, scale), two fp32 tensors of one element on the GPU: the norm of all
    gradients (None is passed over), and the factor min(1, max_norm / (norm + 1e-6))
    that clips them, for the steps' `scale`.  Where the norm is not finite the
    factor is NaN, and a step with it changes nothing.  t: an int64 tensor, a
    count of steps that is raised by one if the norm is finite.  out: fp32 of two
    elements for both."""
    return norm_into(out, grads, max_norm, t, stream).unbind()


def norm_into(out, grads, max_norm, t=None, stream=None):
    """grad_norm's call; `out`, or what is allocated for None."""
    import torch
    grads = _sequence(grads)
    rows, count, index = _native().grads(grads)
    _L.require(count > 0 or out is not None, "there must be a gradient, or out")
    device = _device(index) if count else out.device
    _L.require(device.type == "cuda", "out must be a CUDA tensor")
    L = _L.lib()
    nbytes = L.ma_grad_norm_workspace(count)
    s, place = _stream(device, stream)
    with place:
        if out is None:
            out = torch.empty(2, dtype=torch.float32, device=device)
        to = _state(out, "out", torch.float32, 2, device)
        ws = _workspace(nbytes, device)
        _L.check(L.ma_grad_norm(count, rows, max_norm, to, None if t is None else _one(t, "t", torch.int64, device),
                                ws.data_ptr(), nbytes, s))
    _native().changed((out, t), (), ())
    return out


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
    call = step_call(params, grads, (m, v), t, lr, beta1, beta2, eps, wd, scale, master, stream)
    if call:
        call()


def _moments8(cm, cv, sm, sr, size, device):
    import torch
    return (_state(cm, "cm", torch.int8, size, device), _state(cv, "cv", torch.uint8, size, device),
            _state(sm, "sm", torch.float32, size // BLOCK, device), _state(sr, "sr", torch.float32, size // BLOCK, device))


def step_call(params, grads, state, t, lr, beta1, beta2, eps, wd, scale=None, master=None, stream=None, apart=False):
    """A function that makes the call of adamw_step (state: m, v) or adamw8_step (state: cm,
    cv, sm, sr), after all that is looked at here has been: what a caller who makes several
    of them needs in order to make all or none.  The library itself looks at the
    numbers (check_numbers) and, here with `apart`, at whether parameters
    overlap.  None if there is no gradient."""
    import torch
    params, grads = _sequence(params), _sequence(grads)
    rows, count, index, size = _native().rows(params, grads)
    if not count:
        return None
    device = _device(index)
    if len(state) == 2:
        fn = _L.lib().ma_adamw_many_step
        at = _state(state[0], "m", torch.float32, size, device), _state(state[1], "v", torch.float32, size, device)
    else:
        fn = _L.lib().ma_adamw8_many_step
        at = _moments8(*state, size, device)
    copy = None if master is None else _state(master, "master", torch.float32, size, device)
    a = _arguments(t, lr, beta1, beta2, eps, wd, scale, device)
    if apart:
        _L.require(not _native().overlap(params, grads), "two parameters overlap")
    s, place = _stream(device, stream)

    def call():
        with place:
            _L.check(fn(count, rows, C.byref(a), copy, *at, size, s))
        _native().changed((*state, master), params, grads)

    return call


def adamw8_step(params, grads, cm, cv, sm, sr, t, lr=1e-3, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                wd: float = 0.0, scale=None, master=None, stream=None):
    """adamw_step with the moments in 8 bits: cm int8 and cv uint8 codes of
    state_size(params) elements, sm and sr fp32 scales of one for 256 of them,
    updated in place, all zeros before the first step."""
    call = step_call(params, grads, (cm, cv, sm, sr), t, lr, beta1, beta2, eps, wd, scale, master, stream)
    if call:
        call()


def adamw8_values(cm, cv, sm, sr, stream=None):
    """(m, v), the fp32 moments that an 8-bit state stands for."""
    import torch
    size, device = cm.numel(), cm.device
    _L.require(cm.is_cuda, "cm must be a CUDA tensor")
    _L.require(size % BLOCK == 0, f"cm must have a multiple of {BLOCK} elements")
    state = _moments8(cm, cv, sm, sr, size, device)
    s, place = _stream(device, stream)
    with place:
        m, v = (torch.empty(size, dtype=torch.float32, device=device) for _ in range(2))
        _L.check(_L.lib().ma_adamw8_many_values(size, *state, m.data_ptr(), v.data_ptr(), s))
    return m, v
