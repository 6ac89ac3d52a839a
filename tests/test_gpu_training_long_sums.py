"""Sums over very long axes of terms that are all the same: each addition to a float32 sum of n of them rounds the same way
and may be off by n / 2 * 2^-24 of it, so no sum may be a chain of very many."""
import pytest
import torch

import train_util as tu
from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu
CLOSE = 600 * tu.U  # chains of at most 300 additions, and two of them in a row


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def near(got, want, what, room=CLOSE):
    off = (got.double() - want).abs().max().item()
    assert off <= room * abs(want), f"{what}: off by {off / abs(want):.3g}"


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_layer_norm_of_long_rows(name):
    """One row of 0.1: its mean is 0.1, so y is the bias but for the mean's error times rstd, 1 / sqrt(eps)."""
    dtype, dim = tu.DTYPES[name], (1 << 24) + 3
    x = torch.full((1, dim), 0.1, device="cuda").to(dtype)
    w, b = torch.ones(dim, dtype=dtype, device="cuda"), torch.zeros(dim, dtype=dtype, device="cuda")
    value = x[0, 0].double().item()
    out = binding.gs_layer_norm_fwd(x, w, b, eps=1e-5)
    near(out.mean, value, "mean")
    near(out.rstd, 1e-5 ** -0.5, "rstd", CLOSE + (CLOSE * value) ** 2 / 1e-5)
    assert out.y.abs().max().item() <= CLOSE * value * 1e-5 ** -0.5 * 1.01


def test_layer_norm_gradient_of_long_rows():
    """g = 0.1 and xh = 1 in every column (a mean of the caller's): grad_x = 0.1 - 0.1 - 1 * 0.1 = -0.1."""
    dim = (1 << 24) + 3
    x, g = torch.full((1, dim), 1.0, device="cuda"), torch.full((1, dim), 0.1, device="cuda")
    got = binding.gs_layer_norm_bwd(x, torch.ones(dim, device="cuda"), torch.zeros(1, device="cuda"),
                                    torch.ones(1, device="cuda"), g)
    near(got.x, -g[0, 0].double().item(), "grad x", 3 * CLOSE)


def test_layer_norm_column_sums_of_many_wide_rows():
    rows, dim = 1 << 18, 8200
    x, g = torch.full((rows, dim), 0.7, device="cuda"), torch.full((rows, dim), 0.1, device="cuda")
    w = torch.ones(dim, device="cuda")
    got = binding.gs_layer_norm_bwd(x, w, torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda"), g)
    value = g[0, 0].double().item()
    near(got.bias, rows * value, "grad bias")
    near(got.weight, rows * value * x[0, 0].double().item(), "grad weight")


def test_weight_gradient_of_long_rows():
    dim = 1 << 23
    plan = binding.gs_expert_plan(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1)
    source, g = torch.full((1, dim), 0.7, device="cuda"), torch.full((1, dim), 0.1, device="cuda")
    got = binding.gs_expert_combine_bwd(source, plan, torch.ones(1, 1, device="cuda"), g)
    near(got.weights, dim * source[0, 0].double().item() * g[0, 0].double().item(), "grad weights")
