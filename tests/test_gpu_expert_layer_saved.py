"""What the expert layer keeps for its backward."""
import pytest
import torch

from gpu_util import require_gpu
from tile_binned_gaussian_amd.expert_layer import ExpertLayer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def test_the_logits_are_kept_for_the_route_alone():
    x = torch.randn(50, 16, device="cuda").bfloat16()
    for products in ("library", "f8"):
        for balance in (0.0, 0.1):
            layer = ExpertLayer(16, 8, 4, 2, products=products, balance=balance)
            y, saved = layer.forward(x)
            routed = products == "f8" or balance > 0
            assert (saved.logits is not None) == (saved.route is not None) == routed
            grad_x, grads = layer.backward(saved, torch.ones_like(y))
            assert grad_x.isfinite().all() and set(grads) == set(layer.parameters)
