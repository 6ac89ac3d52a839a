"""How the products of 8-bit rows are summed, as the entry point's contract has it: float32 results of exact products,
16-bit results of products that are cut off 2^-13 below the power of two of the largest of their 8 neighbours."""
import pytest
import torch

import f8_util as fu
import train_util as tu
from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu

# rows x columns below each kernel's tiles: the small and the middle ones
SIZES = [(40, 40), (4500, 1100)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def multiply(x, w, rows, cols, dtype):
    """All rows alike and all columns alike: the one result."""
    qx = binding.gs_quantize(x.expand(rows, -1).contiguous().cuda())
    qw = binding.gs_quantize(w.expand(cols, -1).contiguous().cuda())
    got = binding.gs_expert_product(qx, qw, dtype=dtype)
    assert (got == got[0, 0]).all()
    return got[0, 0].item()


def cancelling(apart):
    """448 * 448 and its opposite in two groups of 8, and 14 products of 15 beside them, or apart in groups of their own."""
    x, w = torch.zeros(256), torch.zeros(256)
    x[0], w[0] = 448.0, 448.0
    x[8], w[8] = 448.0, -448.0
    beside = torch.cat([torch.arange(1, 8), torch.arange(9, 16)])
    at = beside + 16 if apart else beside
    x[at], w[at] = 15.0, 1.0
    return x, w


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("apart", [False, True])
def test_products_that_cancel(rows, cols, apart):
    x, w = cancelling(apart)
    assert multiply(x, w, rows, cols, torch.float32) == 210.0
    want, size, most = fu.product(x.double()[None], w.double()[None, None], torch.tensor([0, 1]))
    for dtype in (torch.bfloat16, torch.float16):
        got = multiply(x, w, rows, cols, dtype)
        if apart:  # no larger product among their 8: whole, 210 in 8 bits too
            assert got == 210.0
        else:
            assert abs(got - 210.0) <= fu.product_bound(want, size, most, 256, dtype).item()


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("place", [0, 3, 7])
def test_the_cut_of_a_group(rows, cols, place):
    """One product of 2^16 and another of its group of 2^(16 - d), alone after the first's opposite in another block: kept
    whole for d up to 13, for float32 results always."""
    for d in range(8, 17):
        x, w = torch.zeros(256), torch.zeros(256)
        x[place], w[place] = 256.0, 256.0
        x[(place + 1) % 8], w[(place + 1) % 8] = 2.0 ** -4, 2.0 ** (20 - d)
        x[136], w[136] = 256.0, -256.0
        want = 2.0 ** (16 - d)
        assert multiply(x, w, rows, cols, torch.float32) == want
        for dtype in (torch.bfloat16, torch.float16):
            got = multiply(x, w, rows, cols, dtype)
            assert got == want if d <= 13 else 0 <= got <= want


def test_float32_results_of_rows_that_cancel():
    """Every row's second half is its first again and the weight's second half the first's opposite, but for one step
    here and there: what is left is summed within float32's bound, of sizes 2^-10 of the terms'."""
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(60, 128, generator=g), torch.randn(70, 128, generator=g)
    less = torch.where(torch.rand(70, 128, generator=g) < 0.02, 1.125, 1.0)
    qx = binding.gs_quantize(torch.cat([x, x], dim=1).cuda())
    qw = binding.gs_quantize(torch.cat([w, -w * less], dim=1).cuda())
    want, size, most = fu.product(fu.held(qx), fu.held(qw)[None], torch.tensor([0, 60]))
    assert want.abs().median() < 0.05 * size.median()
    for dtype in tu.DTYPES.values():
        got = binding.gs_expert_product(qx, qw, dtype=dtype)
        tu.assert_within(got, want, fu.product_bound(want, size, most, 256, dtype), str(dtype))
