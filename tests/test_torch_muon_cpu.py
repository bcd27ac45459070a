"""Argument checks of torch_optim.Muon that need no GPU."""
import pytest
import torch

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
