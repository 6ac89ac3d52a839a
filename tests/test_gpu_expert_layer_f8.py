"""The expert layer on values held in 8 bits, with its balance loss: against the same steps in 64 bits, captured into a
graph, on another stream, and through the rasterizer."""
import os
import sys

import pytest
import torch

import f8_util as fu
import train_util as tu
from gpu_util import require_gpu
from tile_binned_gaussian_amd import synth
from tile_binned_gaussian_amd.expert_layer import ExpertLayer

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def rounded(x):
    """What x [..., dim] stands for when it is held in 8 bits."""
    values, scales = fu.quantize(x)
    return fu.values_of(values, scales, x.shape[-1])


def turned(x):
    return rounded(x.transpose(-1, -2).contiguous())


def steps(layer, x, grad_y, ids):
    """(y, gradients by name) of the layer's steps in 64 bits, each sum and each 8-bit value by its definition."""
    p = {k: v.cpu().double() for k, v in layer.parameters.items()}
    T, K, E = x.shape[0], layer.choices, layer.experts
    n, mean, rstd = tu.layer_norm(x, p["norm_weight"], p["norm_bias"], 1e-5)
    _, w, counts, _, _, kept = fu.route(n @ p["router"], K, ids=ids)
    offsets, rows_of, pairs = tu.expert_plan(ids, E)
    tokens = rounded(n)
    hidden = rounded(fu.product(fu.sorted_rows(tokens, pairs, K), turned(p["up"]), offsets)[0].clamp(min=0))
    rows = fu.product(hidden, turned(p["down"]), offsets)[0]
    y = x.double() + tu.expert_combine(rows, rows_of, w)[0]
    grad_rows, grad_w, _ = tu.expert_combine_grad(rows, rows_of, w, grad_y)
    grads = {"down": fu.weight_grad(hidden, grad_rows, offsets)[0]}
    grad_hidden = fu.product(rounded(grad_rows), rounded(p["down"]), offsets)[0] * (hidden > 0)
    sent = fu.sorted_rows(tokens, pairs, K)
    grads["up"] = fu.weight_grad(sent, grad_hidden, offsets)[0]
    grad_sent = fu.product(rounded(grad_hidden), rounded(p["up"]), offsets)[0]
    grad_logits = fu.route_grad(n @ p["router"], ids, w, counts, kept, grad_w, layer.balance, True)[0]
    grads["router"] = tokens.T @ grad_logits
    grad_norm = tu.expert_combine(grad_sent, rows_of, None)[0] + grad_logits @ p["router"].T
    gx, grads["norm_weight"], grads["norm_bias"] = tu.layer_norm_grad(x, p["norm_weight"], mean, rstd, grad_norm)
    grads["x"] = grad_y.double() + gx
    return y, grads


@pytest.mark.parametrize("tokens,dim,hidden,experts,choices", [(1, 16, 8, 3, 2), (45, 33, 20, 5, 1), (203, 64, 136, 8, 3),
                                                               (300, 140, 64, 4, 4)])
def test_gradients_against_64_bits(tokens, dim, hidden, experts, choices):
    """float32 sums are 8e-4 of a gradient's norm apart at most, as in the layer of library products. They differ by about
    2^-20 of a value, so that about one value in 2^15 lies so near to the middle of two of its 8-bit neighbours (2^-4 apart)
    that it goes to the other one: 2^-4 * 2^-7.5 of the norm, at three places that follow each other."""
    layer = ExpertLayer(dim, hidden, experts, choices, seed=tokens, dtype=torch.float32, products="f8", balance=0.05)
    g = torch.Generator().manual_seed(tokens)
    x, gy = torch.randn(tokens, dim, generator=g), torch.randn(tokens, dim, generator=g)
    layer.parameters["norm_bias"].copy_(0.1 * torch.randn(dim, generator=g))
    y, saved = layer.forward(x.cuda())
    grad_x, grads = layer.backward(saved, gy.cuda())
    want, want_grads = steps(layer, x, gy, saved.route.ids.cpu())
    for name, got, exact in [("y", y, want), ("x", grad_x, want_grads["x"])] + \
            [(k, grads[k], want_grads[k]) for k in layer.parameters]:
        off, size = (got.cpu().double() - exact).norm().item(), exact.norm().item()
        assert off <= (8e-4 + 3 * 2.0 ** -11.5) * size + 1e-12, (name, off, size)


def test_the_balance_loss_joins_library_products():
    """The gradient with a balance loss less that without is the loss's own, for the router's weight and for x."""
    layer = ExpertLayer(32, 16, 6, 2, seed=1, dtype=torch.float32, balance=0.5)
    plain = ExpertLayer(32, 16, 6, 2, seed=1, dtype=torch.float32)
    g = torch.Generator().manual_seed(9)
    x, gy = torch.randn(200, 32, generator=g), torch.randn(200, 32, generator=g)
    (y, saved), (y0, saved0) = layer.forward(x.cuda()), plain.forward(x.cuda())
    torch.testing.assert_close(y, y0, rtol=1e-6, atol=1e-6)
    (gx, grads), (gx0, grads0) = layer.backward(saved, gy.cuda()), plain.backward(saved0, gy.cuda())
    p = {k: v.cpu().double().requires_grad_() for k, v in layer.parameters.items()}
    wide = x.double().requires_grad_()
    n = tu.layer_norm(wide, p["norm_weight"], p["norm_bias"], 1e-5)[0]
    loss = fu.route(n @ p["router"], 2, ids=saved.ids.cpu())[4]
    assert abs(saved.route.loss.item() - loss.item()) < 1e-5
    (0.5 * loss).backward()
    # both gradients are off by roundings of their own size, 2^-24 times a few hundred
    for got, base, want in ((grads["router"], grads0["router"], p["router"].grad), (gx, gx0, wide.grad)):
        off = (got - base).cpu().double() - want
        assert off.norm() <= 1e-4 * want.norm() + 3e-5 * base.norm().item()
    assert set(grads) == set(layer.parameters)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_captured(dtype):
    """Forward and backward in one graph, with weights held before or in it; every replay, with other work between, gives
    what the eager calls give."""
    layer = ExpertLayer(64, 96, 8, 2, dtype=dtype, products="f8", balance=0.01)
    g = torch.Generator().manual_seed(2)
    xs = [torch.randn(500, 64, generator=g).to(dtype).cuda() for _ in range(4)]
    gy = torch.randn(500, 64, generator=g).to(dtype).cuda()

    def step(x):
        y, saved = layer.forward(x)
        return y, saved.route.loss, *layer.backward(saved, gy)
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x)
    for new in xs + xs[:2]:
        x.copy_(new)
        graph.replay()
        want = step(new)
        torch.cuda.synchronize()
        for a, b in zip(got[:3], want[:3]):
            assert torch.equal(a, b)
        for k in got[3]:
            assert torch.equal(got[3][k], want[3][k]), k


def test_on_another_stream_with_weights_held_once():
    layer = ExpertLayer(64, 96, 8, 2, products="f8")
    x = torch.randn(300, 64, device="cuda").bfloat16()
    want, _ = layer.forward(x)
    held = layer.hold_weights()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = []
    for s in streams:
        with torch.cuda.stream(s):
            results.append(layer.forward(x, held)[0])
    torch.cuda.synchronize()
    for r in results:
        assert torch.equal(r, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_example_runs(dtype):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import fit_colors
    finally:
        sys.path.pop(0)
    losses = fit_colors.fit(synth.tiny(), steps=3, dim=64, hidden=64, experts=4, dtype=dtype, products="f8",
                            balance=0.01)
    assert len(losses) == 3 and all(v == v for v in losses)
