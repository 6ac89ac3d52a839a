"""How exact orthogonalised updates of 16-bit types are where the matrix is large: next to 64 bits, the result is off
by its own rounding and by nothing else that counts."""
import pytest
import torch

import train_util as tu
from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def matrix(kind, m, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    if kind == "gaussian":
        return 1e-2 * normal(m, n)
    if kind == "momentum":
        r = min(m, n) // 32
        return torch.mm(normal(m, r), normal(r, n)) * (1e-3 / r ** 0.5) + 3e-4 * normal(m, n)
    if kind == "orthonormal":
        return torch.linalg.qr(normal(max(m, n), min(m, n)))[0].T.contiguous().view(min(m, n), max(m, n))
    assert kind == "rows"  # of very different sizes
    return 1e-2 * normal(m, n) * torch.exp(1.5 * normal(m, 1))


def steps_in_64_bits(u, steps, coefficients):
    with torch.device("cuda"):
        return tu.orthogonalize(u, steps=steps, coefficients=coefficients)


SETTLING = (1.875, -1.25, 0.375)  # moves every singular value to 1 and stays there


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("kind", ["gaussian", "momentum", "orthonormal", "rows"])
@pytest.mark.parametrize("m,n", [(800, 900), (1111, 784)])
def test_the_error_is_the_results_rounding(m, n, kind, name):
    """Operands of 22 bits are off by 2^-22, which is 2^-11 of a float16 result's rounding (2^-14 of bfloat16's). Twelve
    steps with the default coefficients let a singular value's relative error grow by up to 122 (the product of
    f'(s) s / f(s) along its orbit), and by 7 in the mean square; fewer steps and the other coefficients by less. 122 *
    2^-11 is 0.06 of the rounding and, added in squares, 0.18% of it; ten such roundings make 1.8% at the most. The
    rounding's own 2-norm is taken as it is: of the exact result, rounded."""
    dtype = tu.DTYPES[name]
    u = matrix(kind, m, n, m + len(kind)).to(dtype)
    for steps, coefficients in ((5, tu.COEFFICIENTS), (9, tu.COEFFICIENTS), (12, tu.COEFFICIENTS), (12, SETTLING)):
        want = steps_in_64_bits(u, steps, coefficients)
        got = binding.gs_orthogonalize(u, steps=steps, coefficients=coefficients).double()
        own = (want.to(dtype).double() - want).norm().item()
        off = (got - want).norm().item()
        assert off <= 1.02 * own, f"{steps} steps of {coefficients}: {off / own:.3f} of the result's own rounding"
