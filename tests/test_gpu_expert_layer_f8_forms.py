"""The expert layer on values held in 8 bits against its steps in 64 bits, in every type it is made for, with the router's
gradient taken from the loss itself; and captured over many tokens."""
import pytest
import torch

import f8_util as fu
import train_util as tu
from gpu_util import require_gpu
from test_training_host import differences
from tile_binned_gaussian_amd.expert_layer import ExpertLayer

SIZES = [(1, 16, 8, 3, 2), (45, 33, 20, 5, 1), (203, 64, 136, 8, 3), (300, 140, 64, 4, 4)]


def rounded(x):
    """What x [..., dim] stands for when it is held in 8 bits."""
    values, scales = fu.quantize(x)
    return fu.values_of(values, scales, x.shape[-1])


def turned(x):
    return rounded(x.transpose(-1, -2).contiguous())


def steps(p, x, grad_y, ids, choices, balance, dtype):
    """(y, gradients by name, the router's loss as a function of its weight) of the layer's steps in 64 bits, each result
    rounded to the layer's type where the layer stores it."""
    def kept(t):
        return t if dtype == torch.float32 else t.to(dtype).double()
    T, E, K = x.shape[0], p["router"].shape[1], choices
    exact, mean, rstd = tu.layer_norm(x, p["norm_weight"], p["norm_bias"], 1e-5)
    n = kept(exact)

    def routed(router):
        return fu.route(n @ router, K, ids=ids)
    _, w, counts, _, _, count = routed(p["router"])
    offsets, rows_of, pairs = tu.expert_plan(ids, E)
    tokens = rounded(n)
    hidden = rounded(kept(fu.product(fu.sorted_rows(tokens, pairs, K), turned(p["up"]), offsets)[0].clamp(min=0)))
    rows = kept(fu.product(hidden, turned(p["down"]), offsets)[0])
    y = kept(x.double() + kept(tu.expert_combine(rows, rows_of, w)[0]))
    grad_rows, grad_w, _ = tu.expert_combine_grad(rows, rows_of, w, grad_y)
    grad_rows = kept(grad_rows)
    grads = {"down": fu.weight_grad(hidden, grad_rows, offsets)[0]}
    grad_hidden = kept(fu.product(rounded(grad_rows), rounded(p["down"]), offsets)[0]) * (hidden > 0)
    grads["up"] = fu.weight_grad(fu.sorted_rows(tokens, pairs, K), grad_hidden, offsets)[0]
    grad_sent = kept(fu.product(rounded(grad_hidden), rounded(p["up"]), offsets)[0])
    grad_logits = fu.route_grad(n @ p["router"], ids, w, counts, count, grad_w, balance, True)[0]
    grads["router"] = n.T @ grad_logits
    grad_norm = kept(kept(tu.expert_combine(grad_sent, rows_of, None)[0]) + grad_logits @ p["router"].T)
    gx, grads["norm_weight"], grads["norm_bias"] = tu.layer_norm_grad(x, p["norm_weight"], mean, rstd, grad_norm)
    grads["x"] = kept(grad_y.double() + kept(gx))

    def loss(router):
        r = routed(router)
        combined = sum((grad_y.double() * (rows_of[:, k] >= 0)[:, None] * rows[rows_of[:, k].clamp(min=0).long()]
                        ).sum(dim=1) @ r[1][:, k] for k in range(K))
        return combined + balance * r[4]
    return y, grads, loss


def parameters(g, dim, hidden, experts):
    def normal(*shape, std=1.0):
        return std * torch.randn(*shape, generator=g, dtype=torch.float64)
    return {"norm_weight": 1 + normal(dim, std=0.1), "norm_bias": normal(dim, std=0.1),
            "router": normal(dim, experts, std=dim ** -0.5), "up": normal(experts, dim, hidden, std=dim ** -0.5),
            "down": normal(experts, hidden, dim, std=hidden ** -0.5)}


@pytest.mark.parametrize("tokens,dim,hidden,experts,choices", SIZES)
def test_the_router_gradient_against_differences(tokens, dim, hidden, experts, choices):
    """The logits come from the tokens as they are, so the gradient takes those and not their 8-bit values."""
    g = torch.Generator().manual_seed(tokens)
    p = parameters(g, dim, hidden, experts)
    x, gy = torch.randn(tokens, dim, generator=g), torch.randn(tokens, dim, generator=g)
    n = tu.layer_norm(x, p["norm_weight"], p["norm_bias"], 1e-5)[0]
    ids = fu.choose(n @ p["router"], choices)
    _, grads, loss = steps(p, x, gy, ids, choices, 0.05, torch.float32)
    wide = p["router"].clone().requires_grad_()
    loss(wide).backward()
    assert (grads["router"] - wide.grad).norm() <= 1e-10 * wide.grad.norm()
    if dim < 40:
        numeric = differences(loss, p["router"])
        # both losses of an entry are off by some 2^-53 of the sum's terms (|x y| of each token), over 2e-6; one choice's
        # weight is 1 whatever the router, which leaves the balance loss's small gradient beside that
        noise = 2.0 ** -53 * tokens * dim / 1e-6
        assert (numeric - wide.grad).norm() <= 1e-7 * wide.grad.norm() + noise * p["router"].numel() ** 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,dim,hidden,experts,choices", SIZES)
def test_gradients_against_64_bits(tokens, dim, hidden, experts, choices, name):
    """What is kept is held in 8 bits by both, in three places that follow each other. float32: sums are 8e-4 of a norm apart
    at most, as in the layer of library products, and about 2^-20 of a value, so that one value in 2^15 lies so near to the
    middle of two 8-bit neighbours (2^-4 apart) that it goes to the other one: 2^-4 * 2^-7.5 of the norm.
    16 bits: the products' cut is about 2^-16 of a value, and a step of bfloat16 (2^-7) or float16 (2^-10) is the other one
    for a value in 2^8 or 2^5 of these, which is 2^-11.5 or 2^-13 of the norm; and 2^-16 of a step of 8 bits (2^-4 to
    2^-3) goes on as one value in 2^12, each of 2^-3 of itself: 2^-9 of the norm."""
    require_gpu()
    dtype = tu.DTYPES[name]
    layer = ExpertLayer(dim, hidden, experts, choices, seed=tokens, dtype=dtype, products="f8", balance=0.05)
    g = torch.Generator().manual_seed(tokens)
    x, gy = (torch.randn(tokens, dim, generator=g).to(dtype) for _ in range(2))
    layer.parameters["norm_bias"].copy_(0.1 * torch.randn(dim, generator=g))
    y, saved = layer.forward(x.cuda())
    grad_x, grads = layer.backward(saved, gy.cuda())
    p = {k: v.cpu().double() for k, v in layer.parameters.items()}
    want, want_grads, _ = steps(p, x, gy, saved.route.ids.cpu(), choices, layer.balance, dtype)
    near = 8e-4 + 3 * (2.0 ** -11.5 if name == "f32" else 2.0 ** -9 + 2.0 ** -11.5)
    for what, got, exact in [("y", y, want), ("x", grad_x, want_grads["x"])] + \
            [(k, grads[k], want_grads[k]) for k in layer.parameters]:
        off, size = (got.cpu().double() - exact).norm().item(), exact.norm().item()
        assert off <= near * size + 1e-12, (what, off / size)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_captured_over_many_tokens(name):
    """Long sums in the router's gradient, in a graph of forward and backward: every replay, with other work between, gives
    what the eager calls give."""
    require_gpu()
    dtype = tu.DTYPES[name]
    layer = ExpertLayer(64, 96, 8, 2, dtype=dtype, products="f8", balance=0.01)
    g = torch.Generator().manual_seed(2)
    xs = [torch.randn(30000, 64, generator=g).to(dtype).cuda() for _ in range(3)]
    gy = torch.randn(30000, 64, generator=g).to(dtype).cuda()

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
