"""Argument checks of torch_optim.AdamW that need no GPU."""
import pytest
import torch

from memory_compressed_adaptive_amd import torch_optim
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
