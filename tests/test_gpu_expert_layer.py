"""The expert layer that runs the training operators together: its gradients against a 64-bit layer's, and a scene's
colours fitted through the rasterizer."""
import os
import sys

import pytest
import torch

from gpu_util import require_gpu
from tile_binned_gaussian_amd import synth

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def wide_layer(p, x, ids, choices):
    """The layer in 64 bits on the CPU, token by token's chosen experts, differentiable."""
    c = x - x.mean(dim=1, keepdim=True)
    n = c * (c.square().mean(dim=1, keepdim=True) + 1e-5).rsqrt() * p["norm_weight"] + p["norm_bias"]
    weights = (n @ p["router"]).gather(1, ids).softmax(dim=1)
    of = [(n @ p["up"][e]).relu() @ p["down"][e] for e in range(p["up"].shape[0])]
    rows = torch.stack(of, dim=1).gather(1, ids[:, :, None].expand(-1, -1, x.shape[1]))
    return x + (weights[:, :, None] * rows).sum(dim=1)


@pytest.mark.parametrize("tokens,dim,hidden,experts,choices", [(1, 16, 8, 3, 2), (45, 33, 20, 5, 1), (203, 64, 96, 8, 3)])
def test_gradients_against_64_bits(tokens, dim, hidden, experts, choices):
    """In float32 every product is off by at most depth * 2^-24 of |a| |b|, which is at most 16 times |a b| here, and
    four of depth up to 203 follow each other: 2^-24 * 4 * 203 * 16 < 8e-4 of a gradient's norm."""
    from tile_binned_gaussian_amd.expert_layer import ExpertLayer
    layer = ExpertLayer(dim, hidden, experts, choices, seed=tokens, dtype=torch.float32)
    g = torch.Generator().manual_seed(tokens)
    x, gy = torch.randn(tokens, dim, generator=g), torch.randn(tokens, dim, generator=g)
    layer.parameters["norm_bias"].copy_(0.1 * torch.randn(dim, generator=g))
    y, saved = layer.forward(x.cuda())
    grad_x, grads = layer.backward(saved, gy.cuda())
    p = {k: v.cpu().double().requires_grad_() for k, v in layer.parameters.items()}
    wide = x.double().requires_grad_()
    want = wide_layer(p, wide, saved.ids.cpu().long(), choices)
    (want * gy.double()).sum().backward()
    for name, got, exact in [("y", y, want.detach()), ("x", grad_x, wide.grad)] + \
            [(k, grads[k], p[k].grad) for k in p]:
        off, size = (got.cpu().double() - exact).norm().item(), exact.norm().item()
        assert off <= 8e-4 * size + 1e-12, (name, off, size)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_colours_of_a_scene_are_fitted(dtype):
    """The loss of an image falls to a fifth; a wrong sign or a lost gradient would let it rise or stand."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import fit_colors
    finally:
        sys.path.pop(0)
    losses = fit_colors.fit(synth.tiny(), steps=80, dim=64, hidden=64, experts=4, dtype=dtype)
    assert losses[-1] < losses[0] / 5
