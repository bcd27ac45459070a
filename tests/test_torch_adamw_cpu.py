"""Argument checks of torch_optim.AdamW that need no GPU."""
import copy
import ctypes as C
import io
import math
import pickle

import pytest
import torch

from memory_compressed_adaptive_amd import _lib, torch_optim
from memory_compressed_adaptive_amd.torch_optim import AdamW


def _p(*shape, **kw):
    return torch.nn.Parameter(torch.zeros(*shape, **kw))


@pytest.mark.parametrize("shape", [(10, 10), (10,), (2, 3, 4, 5)])
def test_rejects_cpu_parameters(shape):
    with pytest.raises(ValueError, match="CUDA"):
        AdamW([_p(*shape)])


@pytest.mark.parametrize("bits", [4, 16, 0])
def test_rejects_other_state_bits(bits):
    with pytest.raises(ValueError, match="state_bits"):
        AdamW([_p(4)], state_bits=bits)
    with pytest.raises(ValueError, match="state_bits"):
        AdamW([{"params": [_p(4)], "state_bits": bits}])


@pytest.mark.parametrize("norm", [0.0, -1.0, float("nan")])
def test_rejects_a_norm_that_is_not_positive(norm):
    with pytest.raises(ValueError, match="max_norm"):
        AdamW([_p(4)], max_norm=norm)


@pytest.mark.filterwarnings("ignore:optimizer contains")
def test_rejects_a_parameter_given_twice():
    p = _p(4)
    with pytest.raises(ValueError, match="twice"):
        AdamW([p, p])


@pytest.mark.parametrize("error", [ValueError, RuntimeError, torch.OutOfMemoryError, KeyboardInterrupt])
def test_a_group_without_room_for_its_moments_is_not_kept(monkeypatch, error):
    monkeypatch.setattr(torch_optim, "_moments", lambda group, first: {"layout": []})
    opt = AdamW([_p(4, 4)])

    def fails(group, first):
        raise error("no")

    monkeypatch.setattr(torch_optim, "_moments", fails)
    with pytest.raises(error):
        opt.add_param_group({"params": [_p(4, 4)]})
    assert len(opt.param_groups) == 1
    opt.step()          # no gradients: nothing to do
    sd = opt.state_dict()
    assert sd["adamw"]["counts"] == [0] and not any(k.startswith("_") for k in sd["param_groups"][0])


def _part(opt, *missing):
    names = [n for n in "abcdef"[:sum(len(g["params"]) for g in opt.param_groups)]]
    it = iter(names)
    grads = [[None if next(it) in missing else 1 for _ in g["params"]] for g in opt.param_groups]
    used = opt._part(grads)
    opt._begun = True
    for s in used:
        opt._counts[s] += 1
    return used


def test_counts_go_by_the_steps_that_had_a_gradient(monkeypatch):
    monkeypatch.setattr(torch_optim, "_moments", lambda group, first: {"layout": []})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    opt = AdamW([{"params": [_p(1), _p(1), _p(1)]}, {"params": [_p(1)]}])   # a b c, d
    counts = lambda: [int(opt._counts[s]) for g in opt.param_groups for s in g["_slots"]]  # noqa: E731
    assert _part(opt) == [0] and counts() == [1, 1, 1, 1] and opt._histories == 1
    assert _part(opt, "b", "d") == [0] and counts() == [2, 1, 2, 1] and opt._histories == 2
    assert _part(opt) == [0, 1] and counts() == [3, 2, 3, 2]
    assert _part(opt, "a", "b", "c") == [1] and counts() == [3, 2, 3, 3] and opt._histories == 3
    assert _part(opt, "a", "b", "c") == [1] and counts() == [3, 2, 3, 4] and opt._histories == 3
    opt.add_param_group({"params": [_p(1), _p(1)]})                         # e f
    assert counts() == [3, 2, 3, 4, 0, 0] and opt._histories == 4
    for k in range(3):                                                      # a has none, b one, c two, the others three
        _part(opt, *"abcdef"[:k + 1])
    assert counts() == [3, 3, 5, 7, 3, 3] and opt._histories <= 6
    sd = opt.state_dict()
    other = AdamW([{"params": [_p(1), _p(1), _p(1)]}, {"params": [_p(1)]}, {"params": [_p(1), _p(1)]}])
    other.load_state_dict(sd)
    opt = other
    assert counts() == [3, 3, 5, 7, 3, 3]
    _part(opt, "f")
    assert counts() == [4, 4, 6, 8, 4, 3]


def test_a_first_step_without_some_gradients(monkeypatch):
    monkeypatch.setattr(torch_optim, "_moments", lambda group, first: {"layout": []})
    opt = AdamW([_p(1), _p(1)])
    assert _part(opt, "a") == [0] and opt._counts == [1, 0]
    assert _part(opt) == [0, 1] and opt._counts == [2, 1]


def test_a_history_does_not_part_in_a_captured_step(monkeypatch):
    monkeypatch.setattr(torch_optim, "_moments", lambda group, first: {"layout": []})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    opt = AdamW([_p(1), _p(1)])
    _part(opt, "a")                       # nothing to copy yet
    opt = AdamW([_p(1), _p(1)])
    _part(opt)
    with pytest.raises(RuntimeError, match="other parameters have gradients"):
        _part(opt, "a")
    assert opt._counts == [1, 0] and opt.param_groups[0]["_slots"] == [0, 0] and opt._histories == 1


def test_gradients_are_copied_only_where_they_must_be():
    p = _p(4, 6)
    for g, kept in ((torch.ones(4, 6), True), (torch.ones(4, 6, dtype=torch.bfloat16), True), (torch.ones(6, 4).t(), False),
                    (torch.ones(4, 6, dtype=torch.float16), False), (torch.ones(4, 1).expand(4, 6), False),
                    (torch._neg_view(torch.ones(4, 6)), False)):
        got = torch_optim._like(g, p)
        assert (got is g) == kept and got.stride() == p.stride() and torch.equal(got.float(), g.float())
    turned = _p(6, 4).detach().t()
    assert torch_optim._like(torch.ones(4, 6), turned).stride() == turned.stride()
    with pytest.raises(ValueError, match="sparse"):
        torch_optim._like(torch.ones(4, 6).to_sparse(), p)


class _Library:
    """Refuses numbers as the library does, counts what it is asked to do and launches nothing."""

    def __init__(self):
        self.real, self.calls = _lib.lib(), []

    def ma_grad_norm_workspace(self, count):
        return 0

    def ma_grad_norm(self, count, rows, max_norm, out, t, *rest):
        if not max_norm > 0:
            return self.real.ma_grad_norm(0, None, max_norm, None, None, None, 0, None)
        if t:
            C.cast(t, C.POINTER(C.c_int64))[0] += 1
        self.calls.append("norm")
        return 0

    def ma_adamw_many_step(self, count, rows, args, *rest):
        code = self.real.ma_adamw_many_step(0, None, args, None, None, None, 0, None)
        if code == 0:
            self.calls.append("step")
        return code

    def __getattr__(self, name):
        return getattr(self.real, name)


def _without_a_gpu(monkeypatch):
    """The optimizer over CPU parameters, with the library's calls made to a stand-in."""
    from memory_compressed_adaptive_amd import adamw
    native, library = adamw._native(), _Library()

    class Native:
        def rows(self, params, grads):
            return b"", sum(g is not None for g in grads), 0, adamw.state_size(params)

        def grads(self, grads):
            return b"", len(grads), 0

        def stream(self, index):
            return 7

        def changed(self, *lists):
            pass

        def __getattr__(self, name):
            return getattr(native, name)

    def moments(group, first):
        n = adamw.state_size(group["params"])
        return {"layout": [], "m": torch.zeros(n), "v": torch.zeros(n)}

    def one(t, what, dtype, device):
        if t.dtype != dtype or t.numel() != 1:
            raise ValueError(what)
        return t.data_ptr()

    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: empty(*a, **kw))
    monkeypatch.setattr(adamw, "_native", lambda: Native())
    monkeypatch.setattr(adamw, "_state", lambda t, *rest: t.data_ptr())
    monkeypatch.setattr(adamw, "_one", one)
    monkeypatch.setattr(adamw, "_workspace", lambda nbytes, device: empty(nbytes, dtype=torch.uint8))
    monkeypatch.setattr(_lib, "lib", lambda: library)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch_optim, "_moments", moments)
    return library.calls


BAD_NUMBERS = [dict(eps=0.0), dict(eps=math.nan), dict(betas=(1.0, 0.999)), dict(betas=(0.9, -0.1)), dict(betas=(0.9, math.nan)),
               dict(weight_decay=-0.1), dict(weight_decay=math.inf), dict(lr=math.inf), dict(lr=math.nan), dict(eps=1e-40), dict(eps=1e39)]


@pytest.mark.parametrize("bad", BAD_NUMBERS + [dict(lr=torch.ones(1, dtype=torch.float64)), dict(lr=torch.ones(2)), dict(betas=(0.9,)),
                                               dict(eps=None), dict(weight_decay="0.1")])
@pytest.mark.parametrize("max_norm", [None, 1.0])
@pytest.mark.parametrize("histories", [1, 2])
def test_a_refused_step_is_not_counted(monkeypatch, bad, max_norm, histories):
    calls = _without_a_gpu(monkeypatch)
    ps = [_p(4), _p(4), _p(4)]
    opt = AdamW([{"params": ps[:2]}, {"params": ps[2:]}], max_norm=max_norm)
    for p in ps[:1] if histories == 2 else ps:
        p.grad = torch.ones(4)
    opt.step()
    for p in ps:
        p.grad = torch.ones(4)
    calls.clear()
    before = opt.state_dict()["adamw"]["counts"]
    group = opt.param_groups[1]
    kept = {k: group[k] for k in bad}
    group.update(bad)
    for _ in range(2):
        with pytest.raises((ValueError, TypeError)):
            opt.step()
    assert opt.state_dict()["adamw"]["counts"] == before and calls == []
    group.update(kept)
    opt.step()
    assert opt.state_dict()["adamw"]["counts"] == [n + 1 for n in before] and calls.count("step") == 2 + (histories == 2)


def test_a_step_whose_norm_is_refused_is_not_counted(monkeypatch):
    calls = _without_a_gpu(monkeypatch)
    p = _p(4)
    p.grad = torch.ones(4)
    opt = AdamW([p], max_norm=1.0)
    opt.max_norm = -1.0
    with pytest.raises(_lib.MicroAdamError, match="max_norm"):
        opt.step()
    assert opt.state_dict()["adamw"]["counts"] == [0] and calls == []


@pytest.mark.parametrize("max_norm", [None, 1.0])
def test_a_step_of_overlapping_parameters_is_not_counted(monkeypatch, max_norm):
    """Tied after the optimizer was made, as a model's head and embedding may be."""
    calls = _without_a_gpu(monkeypatch)
    ps = [_p(4), _p(4), _p(4)]
    opt = AdamW([{"params": ps[:1]}, {"params": ps[1:]}], max_norm=max_norm)
    for p in ps:
        p.grad = torch.ones(4)
    opt.step()
    calls.clear()
    ps[2].data = ps[1].data
    with pytest.raises(ValueError, match="overlap"):
        opt.step()
    assert opt.state_dict()["adamw"]["counts"] == [1] and calls == []
    ps[2].grad = None            # not written: no overlap
    opt.step()
    ps[2].data, ps[2].grad = torch.zeros(4), torch.ones(4)
    opt.step()
    assert sorted(opt.state_dict()["adamw"]["counts"]) == [2, 3]


@pytest.mark.parametrize("bad", BAD_NUMBERS)
def test_a_group_with_bad_numbers_is_not_kept(monkeypatch, bad):
    monkeypatch.setattr(torch_optim, "_moments", lambda group, first: {"layout": []})
    with pytest.raises(ValueError):
        AdamW([_p(4)], **bad)
    opt = AdamW([_p(4)])
    with pytest.raises(ValueError):
        opt.add_param_group({"params": [_p(4)], **bad})
    assert len(opt.param_groups) == 1


@pytest.mark.parametrize("what", ["lr", "beta1", "beta2", "eps", "wd"])
def test_the_numbers_refused_are_the_librarys(what):
    """The step's look at its numbers and the library's, at both sides of each border."""
    from memory_compressed_adaptive_amd import adamw
    tiny, huge = 2.0 ** -126, float(torch.finfo(torch.float32).max)
    for x in (0.0, -0.0, 1.0, math.nextafter(1.0, 0.0) if hasattr(math, "nextafter") else 1.0 - 2.0 ** -53, tiny, tiny * (1 - 2.0 ** -53), huge,
              huge * (1 + 2.0 ** -52), 1e300, -1e-300, -1.0, math.inf, -math.inf, math.nan, 5e-324, 1, 0):
        kw = {**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.0), what: x}
        code = _lib.lib().ma_adamw_many_step(0, None, C.byref(_lib.AdamwArgs(**kw, t=1)), None, None, None, 0, None)
        try:
            adamw.check_numbers(**kw)
            taken = True
        except ValueError:
            taken = False
        assert taken == (code == 0), (what, x)


def test_a_moved_parameter_is_found():
    from memory_compressed_adaptive_amd import adamw
    p = torch.zeros(3, 4)
    kinds = [p, p.to("meta"), p.bfloat16(), p.t(), p.view(12), torch._neg_view(p)]
    assert len({adamw.layout([x]) for x in kinds}) == len(kinds)
    assert adamw.layout([p]) == adamw.layout([p.clone()])


def test_overlap():
    from memory_compressed_adaptive_amd import adamw
    x, y = torch.zeros(10), torch.zeros(10, dtype=torch.bfloat16)
    overlap = lambda ps, gs=None: adamw._native().overlap(ps, gs or ps)  # noqa: E731
    assert not overlap([]) and not overlap([x]) and not overlap([x[5:], y, x[:5]]) and not overlap([x[3:3], x[:5], x[5:5], x[5:]])
    assert overlap([x, x]) and overlap([x[:5], x[4:]]) and overlap([x[4:], y, x[:5]]) and overlap([x, x[2:3]]) and overlap([y[:6], y[5:]])
    assert not overlap([x, x], [x, None]) and not overlap([x, y, x], [None, y, x])


def test_the_device_is_that_of_the_first_parameter(monkeypatch):
    """Also where the first group is an empty one: counts and norm are on one device."""
    asked = []

    def moments(group, first):
        asked.append(first["params"])
        return {"layout": []}

    monkeypatch.setattr(torch_optim, "_moments", moments)
    p, q = _p(1), _p(2)
    opt = AdamW([{"params": []}, {"params": [p]}, {"params": [q]}])
    opt.add_param_group({"params": [_p(3)]})
    assert [[x is p for x in ps] for ps in asked] == [[], [True], [True], [True]]


def _duplicates():
    def through(dump, load):
        def f(opt):
            buffer = io.BytesIO()
            dump(opt, buffer)
            buffer.seek(0)
            return load(buffer)
        return f
    return [copy.deepcopy, through(pickle.dump, pickle.load), through(torch.save, lambda f: torch.load(f, weights_only=False))]


@pytest.mark.parametrize("duplicate", _duplicates(), ids=["deepcopy", "pickle", "torch.save"])
@pytest.mark.parametrize("max_norm", [None, 1.0])
def test_a_copy_goes_on_by_itself(monkeypatch, duplicate, max_norm):
    calls = _without_a_gpu(monkeypatch)
    opt = AdamW([{"params": [_p(4), _p(4)]}, {"params": [_p(4)]}], max_norm=max_norm)
    opt.param_groups[0]["params"][0].grad = torch.ones(4)
    opt.step()
    other = duplicate(opt)
    assert other.max_norm == max_norm and (other.grad_norm is None) == (max_norm is None)
    assert other.state_dict()["adamw"]["counts"] == opt.state_dict()["adamw"]["counts"] == [1, 0]
    for g in other.param_groups:
        for p in g["params"]:
            p.grad = torch.ones(4)
    calls.clear()
    other.step()
    assert calls.count("step") == 3 and calls.count("norm") == (max_norm is not None)
    assert other.state_dict()["adamw"]["counts"] == [2, 1] and opt.state_dict()["adamw"]["counts"] == [1, 0]
    other.add_param_group({"params": [_p(5)]})
    again = AdamW([{"params": [_p(4), _p(4)]}, {"params": [_p(4)]}, {"params": [_p(5)]}])
    again.load_state_dict(other.state_dict())
    assert again.state_dict()["adamw"]["counts"] == [2, 1, 0]


def test_a_copy_of_an_optimizer_without_parameters(monkeypatch):
    monkeypatch.setattr(torch_optim, "_moments", lambda group, first: {"layout": []})
    opt = copy.deepcopy(AdamW([{"params": []}]))
    opt.add_param_group({"params": [_p(3)]})
    assert opt.state_dict()["adamw"]["counts"] == [0]


def _moments_on_the_cpu(monkeypatch):
    """The real moments, for CPU parameters that say they are CUDA ones where they are looked at."""
    real = torch_optim._moments

    class On:
        """A parameter whose device is of type cuda, and which makes its tensors on the CPU."""

        class device:
            type = "cuda"

        def __init__(self, p):
            self._p = p

        def __getattr__(self, name):
            return getattr(self._p, name)

    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **kw: zeros(*a, **kw))
    monkeypatch.setattr(torch_optim._adamw, "require_dense", lambda ps: None)
    monkeypatch.setattr(torch_optim, "_moments", lambda group, first: real({**group, "params": [On(p) for p in group["params"]]},
                                                                           {"params": [On(p) for p in first["params"]][:0]}))
    return zeros


F32, BF16 = torch.float32, torch.bfloat16


def _filled(dtypes, value, **kw):
    return AdamW([torch.nn.Parameter(torch.full((4, 3), value).to(d)) for d in dtypes], master_weights=True, **kw)


def test_copies_are_of_16_bit_parameters_alone(monkeypatch):
    """Those of others would go stale: no step uses them."""
    _moments_on_the_cpu(monkeypatch)
    master = _filled((BF16, F32), 1.0).param_groups[0]["_moments"]["master"]
    assert bool((master[:12] == 1).all()) and not bool(master[12:].any())


@pytest.mark.parametrize("bits", [32, 8])
def test_load_refuses_types_whose_copies_were_not_kept(monkeypatch, bits):
    """fp32 when saved and bf16 now: the parameter would go on from a copy that no step had written."""
    _moments_on_the_cpu(monkeypatch)
    saved = _filled((BF16, F32), 1.0, state_bits=bits).state_dict()
    now = _filled((BF16, BF16), 5.0, state_bits=bits)
    with pytest.raises(ValueError, match="saved"):
        now.load_state_dict(saved)
    assert bool((now.param_groups[0]["_moments"]["master"][:12] == 5).all())
    for dtypes in ((BF16, F32), (F32, BF16)):
        opt = _filled(dtypes, 5.0, state_bits=bits)
        if dtypes == (F32, BF16):
            with pytest.raises(ValueError, match="saved"):
                opt.load_state_dict(saved)
        else:
            opt.load_state_dict(saved)
            assert bool((opt.param_groups[0]["_moments"]["master"][:12] == 1).all())
    _filled((BF16, F32), 5.0, state_bits=bits).load_state_dict(_filled((BF16, BF16), 1.0, state_bits=bits).state_dict())


def test_load_takes_other_types_without_copies(monkeypatch):
    """Moments are the same in either type."""
    _moments_on_the_cpu(monkeypatch)
    a, b = (AdamW([torch.nn.Parameter(torch.zeros(4, 3, dtype=d))]) for d in (F32, BF16))
    a.param_groups[0]["_moments"]["m"].fill_(3.0)
    b.load_state_dict(a.state_dict())
    assert bool((b.param_groups[0]["_moments"]["m"] == 3).all())


def test_load_takes_states_that_were_saved_without_types(monkeypatch):
    """As this optimizer saved them at first: they are taken to be of the parameters' types now."""
    _moments_on_the_cpu(monkeypatch)
    saved = _filled((BF16, F32), 1.0).state_dict()
    for st in saved["adamw"]["groups"]:
        assert st.pop("types") == ["bfloat16", "float32"]
    opt = _filled((BF16, F32), 5.0)
    opt.load_state_dict(saved)
    assert bool((opt.param_groups[0]["_moments"]["master"][:12] == 1).all())
    assert opt.state_dict()["adamw"]["groups"][0]["types"] == ["bfloat16", "float32"]


def _rated(lr, *more):
    return AdamW([{"params": [_p(4)], "lr": lr}, *({"params": [_p(4)], "lr": x} for x in more)])


@pytest.mark.parametrize("shape", [(1,), ()])
@pytest.mark.parametrize("saved", [0.25, torch.tensor(0.25), torch.tensor([0.25], dtype=torch.float64)], ids=["number", "0-d", "1-d of 64 bits"])
def test_load_writes_a_rate_where_it_lies(monkeypatch, shape, saved):
    """A captured step reads it there."""
    monkeypatch.setattr(torch_optim, "_moments", lambda group, first: {"layout": []})
    rate = torch.full(shape, 0.5)
    opt = _rated(rate, 3.0)
    state = _rated(saved, 2.0).state_dict()
    opt.load_state_dict(state)
    assert opt.param_groups[0]["lr"] is rate and rate.shape == shape and rate.tolist() in (0.25, [0.25])
    assert opt.param_groups[1]["lr"] == 2.0
    rate.fill_(0.125)
    assert float(torch.as_tensor(saved)) == float(torch.as_tensor(state["param_groups"][0]["lr"])) == 0.25


def test_load_takes_a_rate_in_a_tensor_for_a_number(monkeypatch):
    monkeypatch.setattr(torch_optim, "_moments", lambda group, first: {"layout": []})
    rate, opt = torch.tensor([0.25]), _rated(0.5)
    opt.load_state_dict(_rated(rate).state_dict())
    got = opt.param_groups[0]["lr"]
    assert torch.is_tensor(got) and got is not rate and torch.equal(got, rate)


def test_load_into_a_shared_rate(monkeypatch):
    monkeypatch.setattr(torch_optim, "_moments", lambda group, first: {"layout": []})
    rate = torch.tensor([0.5])
    opt = _rated(rate, rate)
    opt.load_state_dict(_rated(0.25, 0.25).state_dict())
    assert all(g["lr"] is rate for g in opt.param_groups) and float(rate) == 0.25
    with pytest.raises(ValueError, match="share"):
        opt.load_state_dict(_rated(0.125, 0.0625).state_dict())
    assert all(g["lr"] is rate for g in opt.param_groups) and float(rate) == 0.25


def _captured(monkeypatch, **kw):
    """An optimizer of a, b (one group) and c, whose second step, of all but c, has been captured."""
    calls = _without_a_gpu(monkeypatch)
    ps = [_p(4), _p(4), _p(4)]
    opt = AdamW([{"params": ps[:2]}, {"params": ps[2:]}], **kw)
    _gradients(ps, 0, 1, 2)
    opt.step()
    _gradients(ps, 0, 1)
    opt.step()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    opt.step()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return opt, ps, calls


def _gradients(ps, *which):
    for i, p in enumerate(ps):
        p.grad = torch.ones_like(p) if i in which else None


@pytest.mark.parametrize("max_norm", [None, 1.0])
def test_parameters_that_a_captured_step_takes_together_stay_together(monkeypatch, max_norm):
    """A replay goes by one count for them, and would take one that another step had left out by a wrong one."""
    opt, ps, calls = _captured(monkeypatch, max_norm=max_norm)
    for which in ((0,), (1, 2)):
        _gradients(ps, *which)
        calls.clear()
        before = opt.state_dict()["adamw"]
        with pytest.raises(RuntimeError, match="captured"):
            opt.step()
        assert calls == [] and {k: opt.state_dict()["adamw"][k] for k in ("counts", "slots")} == {k: before[k] for k in ("counts", "slots")}
    for which in ((0, 1), (2,), (0, 1, 2)):       # all of them, or none
        _gradients(ps, *which)
        opt.step()
    assert opt.state_dict()["adamw"]["slots"] == [[0, 0], [1]]
    new = AdamW([{"params": ps[:2]}, {"params": ps[2:]}])
    new.load_state_dict(opt.state_dict())
    _gradients(ps, 0)
    new.step()
    assert new.state_dict()["adamw"]["slots"] == [[0, 2], [1]]
    copied = copy.deepcopy(opt)
    _gradients([p for g in copied.param_groups for p in g["params"]], 0)
    copied.step()


def test_load_beside_a_captured_step(monkeypatch):
    opt, ps, _ = _captured(monkeypatch)
    opt.load_state_dict(opt.state_dict())
    other = AdamW([{"params": [_p(4), _p(4)]}, {"params": [_p(4)]}])
    with pytest.raises(RuntimeError, match="captured"):
        opt.load_state_dict(other.state_dict())
    assert opt.state_dict()["adamw"]["slots"] == [[0, 0], [1]]
    _gradients(ps, 0, 1)
    opt.step()


def test_gradients_without_memory_are_copied():
    """Zeros that autograd never wrote down."""
    p, g = _p(4, 6), torch._efficientzerotensor((4, 6))
    got = torch_optim._like(g, p)
    assert got is not g and got.data_ptr() and not bool(got.any())


def test_a_shallow_copy_is_refused(monkeypatch):
    """It would step the same moments by counts of its own."""
    monkeypatch.setattr(torch_optim, "_moments", lambda group, first: {"layout": []})
    with pytest.raises(TypeError, match="deepcopy"):
        copy.copy(AdamW([_p(3)]))
