"""Checks of the many-tensor AdamW operators' C ABI, of their Python front and of
the tests' own reference that need no GPU: every call here is refused, or empty,
before a device is touched."""
import ctypes as C
import math
import weakref

import pytest
import torch

import adamw_reference as R
from memory_compressed_adaptive_amd import _lib as L
from memory_compressed_adaptive_amd import adamw

ONE = dict(param=256, grad=1 << 20, n=100, at=0, p_type=0, g_type=0)


def _list(*tensors):
    return (L.Tensor * len(tensors))(*(L.Tensor(**{**ONE, **t}) for t in tensors))


def _args(**kw):
    return L.AdamwArgs(**{**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.0, t=1), **kw})


def _step(bits, tensors=({},), args=None, copy=None, state=None, state_n=256, count=None, **kw):
    a = _args(**kw) if args is None else args
    state = tuple(4096 * (i + 1) for i in range(2 if bits == 32 else 4)) if state is None else state
    fn = L.lib().ma_adamw_many_step if bits == 32 else L.lib().ma_adamw8_many_step
    rows = None if tensors is None else _list(*tensors)
    return fn(len(tensors) if count is None else count, rows, None if a == 0 else C.byref(a), copy, *state, state_n, None)


BAD_LISTS = [
    (dict(n=-1),), (dict(grad=None),), (dict(grad=(1 << 20) + 2),), (dict(grad=(1 << 20) + 1, g_type=1),), (dict(g_type=2),),
    (dict(g_type=-1),)]
BAD_PARAMS = [
    (dict(param=None),), (dict(param=258),), (dict(param=257, p_type=1),), (dict(p_type=3),),
    (dict(at=8),), (dict(at=-256),), (dict(at=256),), (dict(n=257),),
    ({}, dict(param=1024, at=0)),                    # two tensors' states at one place
    (dict(n=1, at=256), dict(param=1024, n=1, at=0)),   # out of order
    ({}, dict(at=256)), ({}, dict(param=256 + 396, at=256)), (dict(param=652), dict(param=256, at=256)),
    (dict(param=1 << 16, n=300), dict(param=256, at=512), dict(param=(1 << 16) + 1196, at=768)),   # overlapping parameters
]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("tensors", BAD_LISTS + BAD_PARAMS)
def test_steps_refuse_lists(bits, tensors):
    assert _step(bits, tensors, state_n=256 * max(1, len(tensors) + (len(tensors) > 2))) == L.MA_EINVAL
    code, msg = L.last_error()
    assert code == L.MA_EINVAL and msg.startswith("ma_adamw")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kw", [
    dict(lr=math.inf), dict(lr=math.nan), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=math.nan),
    dict(eps=0.0), dict(eps=1e-40), dict(eps=math.inf), dict(eps=math.nan), dict(eps=1e39), dict(wd=-0.1), dict(wd=math.inf),
    dict(t=0), dict(t=-3), dict(t_dev=4), dict(lr_dev=2), dict(scale=1), dict(args=0), dict(copy=8), dict(state_n=-256),
    dict(state_n=255), dict(count=-1), dict(tensors=None, count=1)])
def test_steps_refuse_arguments(bits, kw):
    assert _step(bits, **kw) == L.MA_EINVAL


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_refuse_moments(bits):
    count = 2 if bits == 32 else 4
    for i in range(count):
        for bad in (None, 4098):
            state = [4096 * (k + 1) for k in range(count)]
            state[i] = bad
            assert _step(bits, state=state) == L.MA_EINVAL
            assert "moments" in L.last_error()[1]


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_refuse_memory_that_is_written_twice(bits):
    count = 2 if bits == 32 else 4
    apart = [1 << 16, 1 << 17, 1 << 18, 1 << 19][:count]
    for i in range(count):
        for j in range(i):
            state = list(apart)
            state[i] = state[j]
            assert _step(bits, state=state) == L.MA_EINVAL and "overlap" in L.last_error()[1]
        state = list(apart)
        state[i] = 256 + 384       # the parameter's last elements
        assert _step(bits, state=state) == L.MA_EINVAL and "overlap" in L.last_error()[1]
        assert _step(bits, state=apart, copy=apart[i]) == L.MA_EINVAL and "overlap" in L.last_error()[1]
    assert _step(bits, state=apart, copy=256) == L.MA_EINVAL and "overlap" in L.last_error()[1]


@pytest.mark.parametrize("bits", [32, 8])
def test_sizes_past_the_limit(bits):
    assert _step(bits, (dict(n=(1 << 40) + 1),), state_n=1 << 40) == L.MA_EUNSUPPORTED
    assert _step(bits, state_n=1 << 41) == L.MA_EUNSUPPORTED


@pytest.mark.parametrize("bits", [32, 8])
def test_empty_lists_do_nothing(bits):
    assert _step(bits, (), state=(None,) * 4 if bits == 8 else (None,) * 2, state_n=0) == L.MA_OK
    assert _step(bits, (dict(n=0, param=None, grad=None),), state=(None,) * 4 if bits == 8 else (None,) * 2, state_n=0) == L.MA_OK


def _norm(tensors=({},), max_norm=1.0, out=512, t=None, ws=1024, ws_bytes=1 << 30, count=None):
    return L.lib().ma_grad_norm(len(tensors) if count is None else count, _list(*tensors) if tensors is not None else None, max_norm,
                                out, t, ws, ws_bytes, None)


@pytest.mark.parametrize("tensors", BAD_LISTS)
def test_norm_refuses_lists(tensors):
    assert _norm(tensors) == L.MA_EINVAL
    assert L.last_error()[1].startswith("ma_grad_norm")


@pytest.mark.parametrize("kw", [dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=math.nan), dict(out=None), dict(out=514),
                                dict(t=4), dict(ws=None), dict(ws=1028), dict(ws_bytes=8), dict(count=-1), dict(tensors=None, count=1)])
def test_norm_refuses_arguments(kw):
    assert _norm(**kw) == L.MA_EINVAL


def test_norm_workspace():
    ws = L.lib().ma_grad_norm_workspace
    assert ws(0) == ws(-1) == 0 and 0 < ws(1) <= ws(10000) <= 1 << 20


def test_values_refuse():
    fn = L.lib().ma_adamw8_many_values
    ok = [256, 256, 256, 256, 256, 256]
    assert fn(0, *[None] * 6, None) == L.MA_OK
    assert fn(-256, *ok, None) == fn(100, *ok, None) == L.MA_EINVAL
    assert fn(1 << 41, *ok, None) == L.MA_EUNSUPPORTED
    for i in range(6):
        for bad in (None, 258):
            assert fn(256, *ok[:i], bad, *ok[i + 1:], None) == L.MA_EINVAL


def test_layout_of_a_lists_states():
    ps = [torch.zeros(3, 100), torch.zeros(0), torch.zeros(256), torch.zeros(()), torch.zeros(1)]
    assert adamw.starts(ps) == [0, 512, 512, 768, 1024] and adamw.state_size(ps) == 1280
    flat = torch.arange(1280.0)
    got = adamw.views(flat, ps)
    assert [tuple(v.shape) for v in got] == [(3, 100), (0,), (256,), (), (1,)]
    assert float(got[0][2, 99]) == 299 and float(got[2][0]) == 512 and float(got[3]) == 768 and float(got[4][0]) == 1024
    turned = [torch.zeros(4, 6).t()]
    assert float(adamw.views(flat, turned)[0][5, 3]) == 3 * 6 + 5


def test_python_checks_need_no_device():
    p, g, s = [torch.zeros(4)], [torch.zeros(4)], torch.zeros(256)
    for call in (lambda: adamw.adamw_step(p, g, s, s, 1), lambda: adamw.adamw_step(p, [], s, s, 1), lambda: adamw.grad_norm(g),
                 lambda: adamw.grad_norm([]), lambda: adamw.grad_norm([None]),
                 lambda: adamw.adamw8_step(p, g, s, s, s, s, 1), lambda: adamw.adamw8_values(s.to(torch.int8), s, s, s)):
        with pytest.raises(ValueError):
            call()
    adamw.adamw_step([], [], s, s, 1)


def test_the_references_step_is_torchs():
    """torch.optim.AdamW in 64 bits decays first and multiplies: the same to rounding."""
    g = torch.Generator().manual_seed(3)
    p0 = torch.randn(1000, dtype=torch.float64, generator=g)
    p = torch.nn.Parameter(p0.clone())
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
    m, v = torch.zeros_like(p0), torch.zeros_like(p0)
    for t in range(1, 6):
        p.grad = torch.randn(1000, dtype=torch.float64, generator=g)
        p0, m, v, _ = R.step(p0, p.grad, m, v, t, 1e-2, 0.1)
        opt.step()
        assert torch.allclose(p0, p.detach(), rtol=1e-12, atol=1e-14)


def test_the_references_codes_are_the_nearest():
    g = torch.Generator().manual_seed(4)
    m = torch.randn(700, dtype=torch.float64, generator=g) * 10.0 ** torch.randint(-6, 1, (700,), generator=g).double()
    v = (torch.randn(700, dtype=torch.float64, generator=g) * 10.0 ** torch.randint(-5, 1, (700,), generator=g).double()).square()
    m[5] = v[5] = 0.0
    sm, sr = (x.float() for x in R.tops(m, v))
    cm, cv, _ = R.encode(m, v, sm, sr)
    dm, dv = R.decode(cm, cv, sm, sr)
    assert int(cm[5]) == int(cv[5]) == 0 and bool((cv[v > 0] >= 1).all())
    # half the distance of neighbouring codes, at x = s c^2 / n^2: s (2c + 1) / (2 n^2), or the smallest code
    at = torch.arange(700) // R.BLOCK
    assert bool(((dm - m).abs() <= sm.double()[at] * (2 * cm.double().abs() + 1) / 2 / 127 ** 2 * 1.0001).all())
    assert bool(((dv.sqrt() - v.sqrt()).abs() <= sr.double()[at] * (2 * cv.double() + 1) / 2 / 255 ** 2 * 1.0001).all())
    # a tie goes to the larger: 127^2 units, a value of 2.5 (between 1 and 4)
    cm, *_ = R.encode(torch.tensor([127.0 ** 2, 2.5, -2.5, 2.499], dtype=torch.float64), torch.zeros(4, dtype=torch.float64),
                      torch.tensor([127.0 ** 2]), torch.zeros(1))
    assert cm.tolist() == [127, 2, -2, 1]


def test_the_references_scales():
    s = torch.tensor([1.0, 1.0 + 2.0 ** -23, 1.0, 1.0 + 2.0 ** -23, 1.0 + 2.0 ** -22, float("nan"), 1.0])
    top = torch.tensor([1.0, 1.0, 1.0 + 2.0 ** -24, 1.0 + 2.0 ** -24, 1.0 + 2.0 ** -24, float("nan"), float("nan")], dtype=torch.float64)
    assert R.is_rounded(s, top).tolist() == [True, False, True, True, False, True, False]


@pytest.mark.parametrize("handle,given,switched", [(7, None, False), (None, None, True), (7, "stream", True), (None, "stream", True)])
def test_the_tensors_device_is_current_during_a_call(monkeypatch, handle, given, switched):
    """With the tensors' device current, the current stream's handle will do; otherwise, and for
    a stream that is given, the call is made as the Muon operators make theirs."""
    class Native:
        @staticmethod
        def stream(index):
            assert index == 3
            return handle

    class Stream:
        cuda_stream = 11

    monkeypatch.setattr(adamw, "_native", lambda: Native)
    monkeypatch.setattr(adamw, "_place", lambda device, stream: (Stream, ("placed", device, stream)))
    device = torch.device("cuda", 3)
    got = adamw._stream(device, given)
    assert got == ((11, ("placed", device, given)) if switched else (7, adamw._HERE))


@pytest.mark.parametrize("call", ["norm", "step", "step8"])
@pytest.mark.parametrize("of", [list, iter], ids=["list", "iterator"])
def test_what_an_iterator_yields_is_kept_until_the_call_is_made(monkeypatch, call, of):
    """The list that is read holds addresses only: whoever reads it keeps the tensors."""
    alive, seen = [], []

    class Native:
        @staticmethod
        def grads(gs):
            alive.extend(map(weakref.ref, gs))
            return b"", 2, 0

        @staticmethod
        def rows(ps, gs):
            alive.extend([weakref.ref(x) for xs in (ps, gs) for x in xs])
            return b"", 2, 0, 512

        @staticmethod
        def stream(index):
            return 7

        @staticmethod
        def changed(*lists):
            pass

    class Lib:
        ma_grad_norm_workspace = staticmethod(lambda count: 256)

        def __getattr__(self, name):
            def enqueue(*args):
                seen.extend(r() is not None for r in alive)
                return L.MA_OK
            return enqueue

    monkeypatch.setattr(adamw, "_native", lambda: Native)
    monkeypatch.setattr(adamw, "_state", lambda t, *rest: 0)
    monkeypatch.setattr(adamw, "_workspace", lambda nbytes, device: torch.zeros(nbytes, dtype=torch.uint8))
    monkeypatch.setattr(adamw._L, "lib", Lib)
    tensors = lambda: of([torch.zeros(4), torch.zeros(4)])  # noqa: E731
    s = torch.zeros(512)
    if call == "norm":
        adamw.grad_norm(tensors(), out=torch.zeros(2))
    elif call == "step":
        adamw.adamw_step(tensors(), tensors(), s, s, 1)
    else:
        adamw.adamw8_step(tensors(), tensors(), s, s, s, s, 1)
    assert seen == [True] * (2 if call == "norm" else 4)


def test_the_layout_of_what_an_iterator_yields():
    ps = [torch.zeros(3, 100), torch.zeros(7)]
    flat = torch.arange(1024.0)
    assert [v.shape for v in adamw.views(flat[:768], iter(ps))] == [p.shape for p in ps]
    assert adamw.starts(iter(ps)) == [0, 512] and adamw.state_size(iter(ps)) == 768
    assert adamw.layout(iter(ps)) == adamw.layout(ps) and adamw.missing(iter(ps), iter([None, ps[1]])) == 1
    for given in (ps, iter(ps)):
        with pytest.raises(ValueError, match="CUDA"):
            adamw.require_dense(given)


def test_negated_views_are_refused():
    """Such a view's memory holds the values with the other sign (the imaginary part of a conjugate)."""
    x = torch.complex(torch.zeros(256), torch.ones(256)).conj().imag
    x = x.as_strided((128,), (1,))
    assert x.is_neg() and x.is_contiguous()
    with pytest.raises(ValueError, match="m must be"):
        adamw._state(x, "m", torch.float32, 128, x.device)
    with pytest.raises(ValueError, match="scale must be"):
        adamw._one(x[:1], "scale", torch.float32, x.device)
    y = torch.ones(128)
    assert adamw._state(y, "m", torch.float32, 128, y.device) == adamw._one(y[:1], "scale", torch.float32, y.device) == y.data_ptr()
