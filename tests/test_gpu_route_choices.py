"""The router with more choices than a token has lanes (8, 16 or 64 by the number of experts), and with all experts chosen."""
import pytest
import torch

from gpu_util import require_gpu
from test_gpu_route import check, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,K", [(33, 16, 16), (300, 9, 5), (70, 31, 20), (21, 32, 32), (50, 60, 17), (19, 64, 33),
                                   (40, 200, 40), (9, 256, 256), (12, 300, 70), (5, 1000, 65), (4, 2000, 130)])
def test_many_choices(T, E, K, name):
    x, mask, gw = inputs(T, E, K, name, T + E + K)
    for renormalize in (True, False):
        check(x, K, mask, renormalize, gw)
    if E <= 64:  # fewer experts left than choices
        x[torch.rand(T, E, generator=torch.Generator().manual_seed(K)) < 0.6] = float("-inf")
        check(x, K, None, True, gw)
