"""The training operators at the ends of what they take."""
import pytest
import torch

import train_util as tu
from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [3, 64, 77, 200, 513, 1000, 4100, 9001])
def test_gradient_of_a_large_constant_row(dim, name):
    """x is its own mean, so xh = 0 in every column, rstd = 1 / sqrt(eps) and grad_x = rstd (g - mean g): finite, though
    (0 - mean) * rstd is not. 64 columns are whole packs of fewer lanes than share a row."""
    dtype = tu.DTYPES[name]
    g = torch.Generator().manual_seed(dim)
    x = torch.full((3, dim), 2.0 ** 113, dtype=dtype)
    x[1] = torch.randn(dim, generator=g).to(dtype)
    w, gy = (1 + 0.1 * torch.randn(dim, generator=g)).to(dtype), torch.randn(3, dim, generator=g).to(dtype)
    mean, rstd = tu.layer_norm(x, w, None, 1e-17)[1:]
    mean, rstd = mean.float(), rstd.float()  # 2^113 * 3.2e8 is beyond float32
    assert mean[0] == 2.0 ** 113 and (mean[0] * rstd[0]).isinf()
    got = binding.gs_layer_norm_bwd(x.cuda(), w.cuda(), mean.cuda(), rstd.cuda(), gy.cuda())
    want = tu.layer_norm_grad(x, w, mean, rstd, gy)
    bound = tu.layer_norm_grad_bound(x, w, mean, rstd, gy)
    for part, a, b, c in zip(("x", "weight", "bias"), (got.x, got.weight, got.bias), want, bound):
        tu.assert_within(a, b, c, f"grad {part}")


@pytest.mark.parametrize("shape", [(1, 50), (1, 9000), (2000, 1)])
def test_singular_values_up_to_the_limit(shape):
    """A matrix of one row has one singular value, here moved to 10 and near it: A is its square, in one entry."""
    u = torch.randn(shape, generator=torch.Generator().manual_seed(3))
    for limit, steps in ((10.0, 40), (15.0, 60)):
        coefficients = (1.5, -0.5 / limit ** 2, 0.0)  # s -> 1.5 s - 0.5 s^3 / limit^2
        want = tu.orthogonalize(u, steps=steps, coefficients=coefficients)
        assert abs(want.norm().item() - limit) < 1e-6
        got = binding.gs_orthogonalize(u.cuda(), steps=steps, coefficients=coefficients).cpu().double()
        # the fixed point takes the size's errors back; a step's own roundings, at most ten of 2^-22, stay, and
        # the direction's add up over the steps
        assert (got - want).norm().item() <= 10 * 2.0 ** -22 * steps * limit


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("m,n", [(60, 90), (300, 200), (333, 1000)])
def test_a_matrix_far_smaller_than_the_guard(m, n, name):
    """X = update / (|update| + eps) is then about update / eps, with entries far below a half's smallest value."""
    dtype = tu.DTYPES[name]
    g = torch.Generator().manual_seed(m)
    u = torch.randn(m, n, generator=g)
    u = u / u.norm()
    for size, eps in ((1e-3, 1.0), (1e-6, 1.0), (1e-9, 1.0), (1e-11, 1e-2), (1e-17, 1e-7)):
        v = (u * size).to(dtype)
        want = tu.orthogonalize(v, eps=eps)
        got = binding.gs_orthogonalize(v.cuda(), eps=eps).cpu().double()
        own = (want.to(dtype).double() - want).norm().item()
        # five steps of at most ten roundings of 2^-22 that grow as the matrix does
        assert (got - want).norm().item() <= own + 50 * 2.0 ** -22 * want.norm().item(), (size, eps)


@pytest.mark.parametrize("rows,dim", [(5000, 1), (5000, 3), (200000, 7), (1 << 22, 1), (1 << 21, 3)])
def test_column_sums_of_many_narrow_rows(rows, dim):
    """Terms that are all the same round the same way in every addition of a chain: the worst for a long one. A chain is
    at most: a thread's share (768 workgroups take 256 / 7 rows or more at a time), a workgroup's 256 threads, and 64
    to join the workgroups; 8 for the terms."""
    x, gy = torch.full((rows, dim), 0.7), torch.full((rows, dim), 0.1)
    mean, rstd = torch.zeros(rows), torch.ones(rows)  # xh = x
    w = torch.ones(dim)
    got = binding.gs_layer_norm_bwd(x.cuda(), w.cuda(), mean.cuda(), rstd.cuda(), gy.cuda())
    want = tu.layer_norm_grad(x, w, mean, rstd, gy)
    depth = rows / (768 * (256 // 7)) + 256 + 64 + 8
    for part, a, b in (("weight", got.weight, want[1]), ("bias", got.bias, want[2])):
        tu.assert_within(a, b, depth * tu.U * b.abs(), f"grad {part}")


def test_a_row_of_more_columns_than_a_launch_has_threads_for():
    """2^28 + 70 columns: one row, whose column sums are its terms."""
    dim = (1 << 28) + 70
    g = torch.Generator(device="cuda").manual_seed(1)
    x, gy = (torch.randn(1, dim, generator=g, device="cuda").half() for _ in range(2))
    w = torch.ones(dim, dtype=torch.float16, device="cuda")
    got = binding.gs_layer_norm_bwd(x, w, torch.zeros(1, device="cuda"), torch.ones(1, device="cuda"), gy)
    assert torch.equal(got.bias, gy[0])
    assert torch.equal(got.weight, (gy[0].float() * x[0].float()).half())
    # both sums' means are of at most 2^20 terms a thread and far below one, so grad_x is grad_y within a rounding of
    # each of four operations on values below 8, and the means themselves
    s1, s2 = gy.float().mean().abs().item(), (gy.float() * x.float()).mean().abs().item()
    off = (got.x.float() - gy.float()).abs().max().item()
    assert off <= 8 * 2.0 ** -10 + s1 + 8 * s2 + 1e-3
