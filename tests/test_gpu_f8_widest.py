"""Rows of 2^31 - 1 values: tile numbers and ends beyond 32 bits."""
import pytest
import torch

from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu
WIDE = (1 << 31) - 1


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def whole_numbers(n, dtype):
    """[1, n] of -3 to 3, another pattern than any power of two's."""
    out = torch.empty(1, n, dtype=dtype, device="cuda")
    step = 7 * (1 << 22)
    first = (torch.arange(step, device="cuda") % 7 - 3).to(dtype)
    for at in range(0, n, step):
        out[0, at:at + step] = first[:min(step, n - at)]
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weight_gradient_of_the_widest_gradient(dtype):
    q = binding.gs_quantize(torch.full((1, 1), 2.0, device="cuda"))
    grad = whole_numbers(WIDE, dtype)
    out = torch.full((WIDE + 256,), 9.0, device="cuda")
    got = binding.gs_expert_weight_grad(q, grad, out=out[:WIDE].view(1, WIDE))
    assert (out[WIDE:] == 9).all()
    step = 1 << 28
    for at in range(0, WIDE, step):
        assert torch.equal(got[0, at:at + step], grad[0, at:at + step].float() * 2), at


def test_held_and_weight_gradient_of_the_widest_row():
    x = whole_numbers(WIDE, torch.bfloat16)
    q = binding.gs_quantize(x)
    back = binding.gs_dequantize(q, dtype=torch.bfloat16)
    assert torch.equal(back, x)
    del back
    out = torch.full((WIDE + 256,), 9.0, device="cuda")
    got = binding.gs_expert_weight_grad(q, torch.full((1, 1), 2.0, device="cuda"), out=out[:WIDE].view(WIDE, 1))
    assert (out[WIDE:] == 9).all()
    step = 1 << 28
    for at in range(0, WIDE, step):
        assert torch.equal(got[at:at + step, 0], x[0, at:at + step].float() * 2), at
