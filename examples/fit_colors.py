"""Trains a layer of experts to give the colours of a seeded scene's splats from their features, by rendering.

The features hold the colours themselves (and the places), as an encoder's would: the example shows the training path
and that its gradients are right, not what can be learned from less.

Each step: features -> expert layer -> colour head -> gs_rasterize_fwd; the image's squared error against the scene's
own rendering goes back through gs_rasterize_bwd, the head and the layer, and the weights take orthogonalised updates.

    python examples/fit_colors.py [--steps 60] [--scene tiny|200k] [--dtype bf16|f32] [--products library|f8]
                                  [--balance 0.01]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tile_binned_gaussian_amd import binding, frame, synth  # noqa: E402
from tile_binned_gaussian_amd.expert_layer import ColorHead, ExpertLayer  # noqa: E402


def features(ds, dim, seed=0):
    """[N, dim]: random waves of each splat's place and colour, as an encoder of a scene would give."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = torch.tensor([ds.width, ds.height], device="cuda")
    of = torch.cat([ds.means2d[0] / size * 4, ds.colors[0] * 4], dim=1)
    return torch.sin(of @ torch.randn(of.shape[1], dim, generator=g, device="cuda") +
                     6.3 * torch.rand(dim, generator=g, device="cuda"))


def fit(scene, steps, dim=128, hidden=256, experts=8, choices=2, dtype=torch.bfloat16, rate=1e-3, tell=None,
        products="library", balance=0.0):
    """The loss of every step."""
    ds = frame.to_device(scene)
    want = frame.render_frame(ds)
    target, isect, offsets = want.render.render_colors, want.isect, want.isect_offsets
    x = features(ds, dim).to(dtype)
    layer = ExpertLayer(dim, hidden, experts, choices, dtype=dtype, products=products, balance=balance)
    head = ColorHead(dim)
    losses = []
    for step in range(steps):
        y, saved = layer.forward(x)
        colors = head.forward(y)
        image = binding.gs_rasterize_fwd(ds.means2d, ds.conics, colors[None].contiguous(), ds.opacities,
                                         ds.backgrounds, ds.width, ds.height, ds.tile_size, offsets,
                                         isect.flatten_ids, isect.n_isects, ds.alpha_cutoff, ds.alpha_clamp,
                                         ds.transmittance_threshold)
        off = image.render_colors - target
        losses.append(off.square().mean())
        grad = binding.gs_rasterize_bwd(ds.means2d, ds.conics, colors[None].contiguous(), ds.opacities,
                                        ds.backgrounds, ds.width, ds.height, ds.tile_size, offsets, isect.flatten_ids,
                                        image.render_alphas, image.last_ids, off * (2 / off.numel()),
                                        torch.zeros_like(image.render_alphas), n_isects=isect.n_isects,
                                        alpha_cutoff=ds.alpha_cutoff, alpha_clamp=ds.alpha_clamp)
        grad_y, head_grads = head.backward(y, colors, grad.colors[0])
        _, layer_grads = layer.backward(saved, grad_y)
        head.update(head_grads, rate)
        layer.update(layer_grads, rate)
        if tell is not None and step % 10 == 0:
            tell(f"step {step}: loss {losses[-1].item():.6f}")
    return torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--scene", choices=("tiny", "200k"), default="200k")
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    ap.add_argument("--products", choices=("library", "f8"), default="library")
    ap.add_argument("--balance", type=float, default=0.0, help="weight of the experts' balance loss")
    a = ap.parse_args()
    scene = synth.tiny() if a.scene == "tiny" else synth.config2()
    losses = fit(scene, a.steps, dtype=torch.bfloat16 if a.dtype == "bf16" else torch.float32, tell=print,
                 products=a.products, balance=a.balance)
    print(f"loss {losses[0]:.6f} -> {losses[-1]:.6f}")


if __name__ == "__main__":
    main()
