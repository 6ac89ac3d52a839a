"""What the expert layer refuses (no GPU)."""
import pytest
import torch

from tile_binned_gaussian_amd.expert_layer import ExpertLayer


@pytest.mark.parametrize("asked,given", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32),
                                         (torch.float16, torch.bfloat16)])
def test_features_of_another_type_than_the_layers(asked, given):
    """The type the layer was made for is the one it computes in; features of another one would change it silently."""
    layer = ExpertLayer(16, 8, 3, 2, device="cpu", dtype=asked)
    with pytest.raises(TypeError, match="x must be"):
        layer.forward(torch.zeros(5, 16, dtype=given))
