"""Checks of the Muon operators' C ABI and of the tests' own reference that need
no GPU: every call here is refused, or empty, before a device is touched."""
import ctypes as C
import math

import pytest
import torch

import muon_reference as R
from memory_compressed_adaptive_amd import _lib as L
from memory_compressed_adaptive_amd import muon

OK = (3.4445, -4.7750, 2.0315)


def _k(*triples):
    return (C.c_float * (3 * len(triples)))(*(v for t in triples for v in t))


def _orth(batch=1, rows=4, cols=4, x=256, x_type=0, strides=(4, 16), out=512, ostrides=(4, 16), steps=1, k=None, eps=1e-7,
          ws=1024, ws_bytes=1 << 30):
    k = _k(*([OK] * max(steps, 1))) if k is None else k
    return L.lib().ma_orthogonalize(batch, rows, cols, x, x_type, *strides, out, *ostrides, steps, k, eps, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), L.MA_EINVAL), (dict(rows=-1), L.MA_EINVAL), (dict(cols=-4), L.MA_EINVAL),
    (dict(rows=1 << 20, cols=1 << 14), L.MA_EUNSUPPORTED),
    (dict(rows=(1 << 62), cols=(1 << 62)), L.MA_EUNSUPPORTED),
    (dict(steps=0), L.MA_EINVAL), (dict(steps=65), L.MA_EINVAL), (dict(eps=0.0), L.MA_EINVAL),
    (dict(eps=math.nan), L.MA_EINVAL), (dict(eps=math.inf), L.MA_EINVAL),
    (dict(x=None), L.MA_EINVAL), (dict(out=None), L.MA_EINVAL), (dict(ws=None), L.MA_EINVAL),
    (dict(ws=1025), L.MA_EINVAL), (dict(ws_bytes=16), L.MA_EINVAL), (dict(x=258), L.MA_EINVAL), (dict(out=513), L.MA_EINVAL),
    (dict(x_type=2), L.MA_EINVAL), (dict(x_type=-1), L.MA_EINVAL),
    (dict(strides=(-4, 16)), L.MA_EINVAL), (dict(ostrides=(3, 16)), L.MA_EINVAL),
    (dict(batch=2, ostrides=(4, 15)), L.MA_EINVAL), (dict(batch=2, ostrides=(4, 0)), L.MA_EINVAL),
    (dict(k=_k((math.inf, 0.0, 0.0))), L.MA_EINVAL),
    (dict(k=_k((16.0, 0.0, 0.0))), L.MA_EINVAL),          # P passes 15
    (dict(k=_k((2.0, 0.0, 0.0))), L.MA_EINVAL),           # X passes 1.95
    (dict(k=_k((3.0, -0.3, 0.0))), L.MA_EINVAL),
    (dict(k=_k((0.0, 0.0, 0.0))), L.MA_EINVAL),           # everything vanishes
])
def test_orthogonalize_refuses(kw, code):
    assert _orth(**kw) == code
    got, msg = L.last_error()
    assert got == code and msg.startswith("ma_orthogonalize")


def test_coefficients_are_checked_through_every_step():
    # each is fine alone; 1.9 leaves values that the second then carries past 1.95
    assert _orth(rows=0, k=_k((1.9, 0.0, 0.0))) == L.MA_OK
    assert _orth(rows=0, steps=2, k=_k((1.9, 0.0, 0.0), (1.9, 0.0, 0.0))) == L.MA_EINVAL
    # an extreme inside the interval: s (2.8 - 2.8 s^2) is largest at s = 0.577
    assert _orth(rows=0, k=_k((2.8, -2.8, 0.0))) == L.MA_OK
    assert _orth(rows=0, k=_k((5.4, -5.4, 0.0))) == L.MA_EINVAL


@pytest.mark.parametrize("a,b,ok", [(6.0, -5.0, False), (14.0, -13.0, False), (2.8, -2.8, True), (-6.0, 5.0, False)])
@pytest.mark.parametrize("c", [0.0, 1e-12, 1e-16, -1e-16, 1e-18, -1e-18, 1e-20, -1e-20, 1e-30, -1e-30])
def test_a_tiny_last_coefficient_hides_no_extreme(a, b, ok, c):
    """s (6 - 5 s^2 + c s^4) reaches 2.53 at s = 0.632, however small c is."""
    assert _orth(rows=0, k=_k((a, b, c))) == (L.MA_OK if ok else L.MA_EINVAL)


@pytest.mark.parametrize("kw", [dict(batch=0), dict(rows=0), dict(cols=0)])
def test_empty_batches_do_nothing(kw):
    assert _orth(x=None, out=None, ws=None, ws_bytes=0, **kw) == L.MA_OK


def _step(fn, momentum, batch=1, rows=4, cols=4, params=256, kind=0, ps=(4, 16), grads=512, gs=(4, 16), lr=0.1, beta=0.9,
          wd=0.0, scale=1.0, steps=1, ws=1024, ws_bytes=1 << 30):
    return fn(batch, rows, cols, params, kind, *ps, grads, *gs, *momentum, lr, beta, wd, scale, 1, steps, _k(*([OK] * steps)),
              1e-7, ws, ws_bytes, None)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kw", [
    dict(batch=-1), dict(params=None), dict(grads=None), dict(params=258), dict(grads=513), dict(kind=7), dict(ps=(3, 16)),
    dict(ps=(0, 16)), dict(batch=2, ps=(4, 8)), dict(gs=(-1, 16)), dict(lr=math.inf), dict(beta=1.0), dict(beta=-0.1),
    dict(beta=math.nan), dict(wd=-0.1), dict(wd=math.nan), dict(scale=math.nan), dict(ws=None), dict(ws_bytes=1),
    dict(momentum=None)])
def test_steps_refuse(bits, kw):
    kw = dict(kw)
    fn = L.lib().ma_muon_step if bits == 32 else L.lib().ma_muon8_step
    momentum = (2048,) if bits == 32 else (2048, 4096)
    if "momentum" in kw:
        del kw["momentum"]
        momentum = (None,) * len(momentum)
    assert _step(fn, momentum, **kw) == L.MA_EINVAL
    assert L.last_error()[1].startswith("ma_muon")


def test_momentum8_values_refuses():
    fn = L.lib().ma_momentum8_values
    assert fn(-1, 4, 256, 512, 1024, None) == L.MA_EINVAL
    assert fn(4, -1, 256, 512, 1024, None) == L.MA_EINVAL
    assert fn(0, 4, None, None, None, None) == L.MA_OK
    assert fn(4, 4, None, 512, 1024, None) == L.MA_EINVAL
    assert fn(4, 4, 256, 513, 1024, None) == L.MA_EINVAL
    assert fn(4, 4, 256, 512, 1026, None) == L.MA_EINVAL
    assert fn(1 << 40, 1 << 40, 256, 512, 1024, None) == L.MA_EUNSUPPORTED


def test_workspace_sizes():
    ws = L.lib().ma_orthogonalize_workspace
    assert ws(0, 4, 4) == 0 and ws(1, 0, 4) == 0 and ws(-1, 4, 4) == 0 and ws(1, 1 << 40, 1 << 40) == 0
    assert 0 < ws(1, 4, 4)
    # a long batch is cut into runs: the workspace does not grow without bound
    assert ws(4096, 4096, 4096) < 1 << 30


def test_python_checks_need_no_device():
    cpu = torch.zeros(4, 4)
    for call in (lambda: muon.orthogonalize(cpu), lambda: muon.muon_step(cpu, cpu.bfloat16(), cpu),
                 lambda: muon.momentum8_values(cpu.to(torch.int8), torch.zeros(4, 1))):
        with pytest.raises(ValueError):
            call()
    assert muon.scales_shape((3, 256)) == (3, 1) and muon.scales_shape((2, 3, 257)) == (2, 3, 2)
    assert muon.rms_scale(100, 400) == pytest.approx(4.0)


@pytest.mark.parametrize("current_device,given,switched", [(0, None, False), (1, None, True), (0, 7, True), (1, 7, True)])
def test_the_streams_device_is_current_during_a_call(monkeypatch, current_device, given, switched):
    """The default stream of a device is the null stream there: the call has to be
    made with that device current."""
    class Stream:
        def __init__(self, device, number):
            self.device, self.number = device, number

        def __eq__(self, other):
            return (self.device, self.number) == (other.device, other.number)

    device = torch.device("cuda", 0)
    entered = []

    class Context:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            entered.append(self.s)

        def __exit__(self, *a):
            entered.append(None)

    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(device, 0))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current_device)
    monkeypatch.setattr(torch.cuda, "stream", Context)
    s, place = muon._place(device, None if given is None else Stream(device, given))
    assert s == Stream(device, given or 0)
    with place:
        assert entered == ([s] if switched else [])
    with pytest.raises(ValueError):
        muon._place(device, Stream(torch.device("cuda", 1), 0))


def test_reference_agrees_with_the_singular_values():
    """The reference's products against its meaning: the same scalar polynomial on
    every singular value, with the singular vectors kept."""
    g = torch.Generator().manual_seed(1)
    for shape in ((12, 30), (30, 12), (1, 5)):
        u = torch.randn(shape, generator=g, dtype=torch.float64)
        x, err = R.orthogonalized(u)
        left, s, right = torch.linalg.svd(u / u.norm(), full_matrices=False)
        a, b, c = (float(v) for v in torch.tensor(R.COEFFICIENTS, dtype=torch.float32))
        for _ in range(5):
            s = s * (a + b * s ** 2 + c * s ** 4)
        assert torch.allclose(x, left @ torch.diag(s) @ right, rtol=0, atol=1e-12)
        assert 0 < err < 0.02 * x.norm().item()


def test_reference_bound_holds_for_roundings_made_on_the_cpu():
    """The bound against products whose X, A and P are rounded to fp16 here, and
    against a planted mistake, which it must not let through."""
    g = torch.Generator().manual_seed(2)
    half = lambda t, s: (t * s).half().double() / s  # noqa: E731
    for shape in ((64, 64), (96, 200), (16, 40)):
        u = torch.randn(shape, generator=g, dtype=torch.float64)
        want, err = R.orthogonalized(u)
        for mistake, pairs in ((False, False), (True, False), (False, True)):
            x = half(u / u.norm(), 2.0 ** 14)
            if pairs:
                a, b, c = R.COEFFICIENTS
                eye = torch.eye(len(x), dtype=torch.float64)
                for two in (True, False, True):
                    gram = half(x @ x.T, 2.0 ** 14)
                    p1 = p2 = half(a * eye + b * gram + c * gram @ gram, 2.0 ** 12)
                    if two:
                        t = half(p1 @ gram, 2.0 ** 12)
                        gram = half(t @ p1, 2.0 ** 14)
                        p2 = half(half(a * eye + b * gram + c * gram @ gram, 2.0 ** 12) @ p1, 2.0 ** 8)
                    x = half(p2 @ x, 2.0 ** 14)
                assert (x - want).norm().item() <= err
                continue
            for _ in range(5):
                a, b, c = R.COEFFICIENTS
                gram = half(x @ x.T, 2.0 ** 14)
                if mistake:
                    gram[-8:, :8] = 0              # a piece of the mirror image forgotten
                x = half(a * torch.eye(len(x), dtype=torch.float64) + b * gram + c * gram @ gram, 2.0 ** 12) @ x
                x = half(x, 2.0 ** 14)
            off = (x - want).norm().item()
            assert (off > err) if mistake else (off <= err)


@pytest.mark.parametrize("rows,cols,row,bat,batch,ok", [
    (768, 64, 768, 64, 12, True), (768, 64, 767, 64, 12, False),       # heads as column blocks of one matrix
    (5, 4, 13, 4, 3, True), (5, 4, 12, 4, 3, True), (5, 4, 11, 4, 3, False), (5, 4, 12, 3, 3, False),
    (5, 4, 100, 7, 3, True), (1, 4, 0, 4, 3, True), (5, 4, 4, 20, 3, True), (5, 4, 4, 19, 3, False), (5, 4, 4, 0, 1, True),
    (2, 1 << 20, 1 << 62, 1 << 40, 1 << 30, False)])
def test_written_matrices_may_interleave_but_not_overlap(rows, cols, row, bat, batch, ok):
    """Whole matrices one after the other, or the rows of all matrices side by
    side.  Every call is refused in the end, for its null momentum."""
    assert _step(L.lib().ma_muon_step, (None,), batch=batch, rows=rows, cols=cols, ps=(row, bat), gs=(0, 0), ws_bytes=1 << 60) == L.MA_EINVAL
    assert ("momentum" in L.last_error()[1]) == ok, L.last_error()[1]
    assert ok or "overlap" in L.last_error()[1]


@pytest.mark.parametrize("given", [((1.5, -0.5, 0.0), (2.0, -1.0, 0.0)), [[1.5, -0.5, 0.0], [2.0, -1.0, 0.0]],
                                   ([1.5, -0.5, 0.0], [2.0, -1.0, 0.0]), [(1.5, -0.5, 0.0), (2.0, -1.0, 0.0)],
                                   torch.tensor([[1.5, -0.5, 0.0], [2.0, -1.0, 0.0]])])
def test_coefficients_may_be_any_sequences(given):
    assert list(muon._coefficients(given, 2)) == [1.5, -0.5, 0.0, 2.0, -1.0, 0.0]


@pytest.mark.parametrize("given", [(1.5, -0.5, 0.0), [1.5, -0.5, 0.0], torch.tensor([1.5, -0.5, 0.0])])
def test_one_triple_serves_every_step(given):
    assert list(muon._coefficients(given, 2)) == [1.5, -0.5, 0.0] * 2


@pytest.mark.parametrize("given", [(), [], ((),), (1.0, 2.0), ((1.0, 2.0),), ((1.0, 2.0, 3.0),), ((1.0, 2.0, 3.0), 1.0)])
def test_other_coefficients_are_refused(given):
    with pytest.raises(ValueError, match="coefficients"):
        muon._coefficients(given, 2)


def test_coefficients_that_change_are_read_again():
    a = torch.tensor(1.5)
    assert muon._coefficients((a, -0.5, 0.0), 1)[0] == 1.5
    a += 0.25
    assert muon._coefficients((a, -0.5, 0.0), 1)[0] == 1.75
