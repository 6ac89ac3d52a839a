"""What the expert layer's 8-bit products and balance loss refuse (no GPU)."""
import pytest
import torch

from tile_binned_gaussian_amd.expert_layer import ExpertLayer


def test_unknown_products_and_a_negative_balance():
    with pytest.raises(ValueError, match="products must be"):
        ExpertLayer(16, 8, 3, 2, device="cpu", products="bf16")
    for balance in (-0.1, float("nan")):
        with pytest.raises(ValueError, match="balance must be"):
            ExpertLayer(16, 8, 3, 2, device="cpu", balance=balance)
    with pytest.raises(ValueError, match="weights go with"):
        ExpertLayer(16, 8, 3, 2, device="cpu").forward(torch.zeros(5, 16, dtype=torch.bfloat16), weights=())
