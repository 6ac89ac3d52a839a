"""Whole numbers that leave the C ABI's 32 bits are refused; cut to 32 bits they would be others that it takes."""
import pytest
import torch

from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("steps", [(1 << 32) + 5, -(1 << 32) + 5, 1 << 31])
def test_steps(steps):
    u = torch.ones(20, 30, device="cuda")
    with pytest.raises(ValueError, match="steps"):
        binding.gs_orthogonalize(u, steps=steps)


@pytest.mark.parametrize("experts", [(1 << 32) + 8, 1 << 31])
def test_experts(experts):
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="experts"):
        binding.gs_expert_plan(ids, experts)
