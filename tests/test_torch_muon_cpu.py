"""Argument checks of torch_optim.Muon that need no GPU."""
import pytest
import torch

from memory_compressed_adaptive_amd import torch_optim
from memory_compressed_adaptive_amd.torch_optim import Muon


@pytest.mark.parametrize("shape", [(10, 10), (10,), (2, 3, 4, 5), (2, 3, 4)])
def test_rejects_cpu_parameters_and_other_shapes(shape):
    with pytest.raises(ValueError):
        Muon([torch.nn.Parameter(torch.zeros(shape))])


def test_rejects_other_momentum_bits():
    with pytest.raises(ValueError):
        Muon([torch.nn.Parameter(torch.zeros(4, 4))], momentum_bits=4)


def test_rejects_a_groups_other_momentum_bits():
    with pytest.raises(ValueError, match="momentum_bits"):
        Muon([{"params": [torch.nn.Parameter(torch.zeros(4, 4))], "momentum_bits": 16}])


@pytest.mark.filterwarnings("ignore:optimizer contains")
def test_rejects_a_parameter_given_twice():
    p = torch.nn.Parameter(torch.zeros(4, 4))
    with pytest.raises(ValueError, match="twice"):
        Muon([p, p])


@pytest.mark.parametrize("error", [ValueError, RuntimeError, torch.OutOfMemoryError, KeyboardInterrupt])
def test_a_group_that_cannot_be_laid_out_is_not_kept(monkeypatch, error):
    """Whatever stops it, memory running out above all: the optimizer stays as it
    was and goes on with the groups it has."""
    monkeypatch.setattr(torch_optim, "_stacks", lambda group: [])
    opt = Muon([torch.nn.Parameter(torch.zeros(4, 4))])

    def fails(group):
        raise error("no")

    monkeypatch.setattr(torch_optim, "_stacks", fails)
    with pytest.raises(error):
        opt.add_param_group({"params": [torch.nn.Parameter(torch.zeros(4, 4))]})
    assert len(opt.param_groups) == 1
    opt.step()
    opt.state_dict()
