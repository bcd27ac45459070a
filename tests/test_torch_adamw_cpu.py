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
    assert sd["adamw"]["count"] == 0 and "_moments" not in sd["param_groups"][0]


def test_gradients_are_copied_only_where_they_must_be():
    p = _p(4, 6)
    for g, kept in ((torch.ones(4, 6), True), (torch.ones(4, 6, dtype=torch.bfloat16), True), (torch.ones(6, 4).t(), False),
                    (torch.ones(4, 6, dtype=torch.float16), False), (torch.ones(4, 1).expand(4, 6), False)):
        got = torch_optim._like(g, p)
        assert (got is g) == kept and got.stride() == p.stride() and torch.equal(got.float(), g.float())
    turned = _p(6, 4).detach().t()
    assert torch_optim._like(torch.ones(4, 6), turned).stride() == turned.stride()
    with pytest.raises(ValueError, match="sparse"):
        torch_optim._like(torch.ones(4, 6).to_sparse(), p)
