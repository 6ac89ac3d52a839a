"""A layer of experts over splat features, trained through the library's entry points.

``ExpertLayer`` is a residual layer, y = x + experts(layer norm(x)): a router picks each token's best experts, the
tokens are sorted by expert, every expert is a two-layer perceptron on its own rows, and the weighted results return
to their tokens. The backward is written out call by call; weight matrices move by their orthogonalised momentum.
The experts' own products are plain library products, one per expert and direction, or with ``products="f8"`` the
library's own on values held in 8 bits: the tokens and the hidden values are then kept for the backward in 8 bits, no row
is copied into sorted order, and nothing waits for the host, so the layer can be captured into a graph. The router's
projection and its gradients are plain products of the tokens as they are either way. ``ColorHead`` maps features to
colours in (0, 1). Both keep float32 parameters; the layer computes in the type it is made for, the head in float32.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import binding


def _normal(g, *shape, std):
    return torch.randn(*shape, generator=g, device=g.device) * std


class _Momentum:
    """Parameters by name with their momentum; matrices ([m, n] or [experts, m, n]) take orthogonalised updates."""

    def __init__(self, parameters):
        self.parameters = parameters
        self._momentum = {k: torch.zeros_like(p) for k, p in parameters.items()}

    def update(self, grads, rate, decay=0.9):
        """momentum = decay momentum + gradient; a matrix moves by rate times its orthogonalised momentum, scaled to
        entries of one size whatever its shape, a vector by rate times its momentum's sign."""
        for name, p in self.parameters.items():
            m = self._momentum[name].mul_(decay).add_(grads[name])
            if p.dim() == 1:
                p.add_(torch.sign(m), alpha=-rate)
            else:
                p.add_(binding.gs_orthogonalize(m), alpha=-rate * max(p.shape[-2:]) ** 0.5)


@dataclass
class _Saved:
    x: torch.Tensor
    norm: binding.LayerNorm
    plan: binding.ExpertPlan
    bounds: list  # the plan's offsets on the host
    ids: torch.Tensor
    weights: torch.Tensor
    sent: torch.Tensor
    hidden: torch.Tensor  # the experts' hidden values after the rectifier, in sorted rows
    rows: torch.Tensor  # the experts' results, in sorted rows
    logits: torch.Tensor | None  # with a balance loss, as the route
    route: binding.ExpertRoute | None


@dataclass
class HeldWeights:
    """The experts' weights in 8 bits, along the sums of the forward and of the backward."""
    up: binding.Quantized  # [experts, hidden, dim]
    down: binding.Quantized  # [experts, dim, hidden]
    up_back: binding.Quantized  # [experts, dim, hidden]
    down_back: binding.Quantized  # [experts, hidden, dim]


@dataclass
class _SavedHeld:
    x: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor
    logits: torch.Tensor
    route: binding.ExpertRoute
    plan: binding.ExpertPlan
    weights: HeldWeights
    tokens: binding.Quantized  # the normalised tokens
    hidden: binding.Quantized  # the experts' hidden values after the rectifier, in sorted rows


class ExpertLayer(_Momentum):
    """products: "library" or "f8". balance: the weight of the balance loss, whose gradient the backward adds to that of
    the result; the forward's loss is then saved.route.loss (library products without a balance loss route in plain torch
    operations: saved.route is None)."""

    def __init__(self, dim, hidden, experts, choices, seed=0, device="cuda", dtype=torch.bfloat16, products="library",
                 balance=0.0):
        if products not in ("library", "f8"):
            raise ValueError(f'products must be "library" or "f8" (got {products!r})')
        if not balance >= 0:
            raise ValueError(f"balance must be >= 0 (got {balance})")
        g = torch.Generator(device=device).manual_seed(seed)
        self.experts, self.choices, self.dtype, self.hidden = experts, choices, dtype, hidden
        self.products, self.balance = products, float(balance)
        self._grad_loss = torch.full((), self.balance, device=device) if balance else None
        super().__init__({"norm_weight": torch.ones(dim, device=device), "norm_bias": torch.zeros(dim, device=device),
                          "router": _normal(g, dim, experts, std=dim ** -0.5),
                          "up": _normal(g, experts, dim, hidden, std=dim ** -0.5),
                          "down": _normal(g, experts, hidden, dim, std=hidden ** -0.5)})

    def _of_experts(self, rows, weight, bounds, out):
        """rows @ weight[e] for every expert's rows; the rows past the kept ones become zeros."""
        for e in range(self.experts):
            if bounds[e + 1] > bounds[e]:
                torch.mm(rows[bounds[e]:bounds[e + 1]], weight[e], out=out[bounds[e]:bounds[e + 1]])
        out[bounds[-1]:].zero_()
        return out

    def hold_weights(self):
        """The experts' weights as they are now in 8 bits, for calls of forward until the next update."""
        up, down = self.parameters["up"], self.parameters["down"]
        return HeldWeights(binding.gs_quantize(up, transpose=True), binding.gs_quantize(down, transpose=True),
                           binding.gs_quantize(up), binding.gs_quantize(down))

    def _forward_held(self, x, weights):
        p = self.parameters
        weights = self.hold_weights() if weights is None else weights
        norm = binding.gs_layer_norm_fwd(x, p["norm_weight"], p["norm_bias"])
        logits = norm.y.float() @ p["router"]
        route = binding.gs_expert_route(logits, self.choices)
        plan = binding.gs_expert_plan(route.ids, self.experts)
        tokens = binding.gs_quantize(norm.y)
        hidden = binding.gs_quantize(binding.gs_expert_product(tokens, weights.up, plan, gather=True, relu=True,
                                                               dtype=x.dtype))
        rows = binding.gs_expert_product(hidden, weights.down, plan, dtype=x.dtype)
        y = x + binding.gs_expert_combine(rows, plan, route.weights)
        return y, _SavedHeld(x, norm.mean, norm.rstd, logits, route, plan, weights, tokens, hidden)

    def _backward_held(self, s, grad_y):
        """The experts' results are formed again from the hidden values kept. Gradients of 8-bit values are those of the
        values that they stand for (a hidden value that rounds to 0 passes none on); the output gradients of both products
        are held in 8 bits too, for the gradients of their inputs. The router's logits are of the tokens themselves, and so
        is its weight's gradient: they are normalised again."""
        p, t = self.parameters, s.x.dtype
        rows = binding.gs_expert_product(s.hidden, s.weights.down, s.plan, dtype=t)
        combine = binding.gs_expert_combine_bwd(rows, s.plan, s.route.weights, grad_y)
        grads = {"down": binding.gs_expert_weight_grad(s.hidden, combine.rows, s.plan)}
        grad_hidden = binding.gs_expert_product(binding.gs_quantize(combine.rows), s.weights.down_back, s.plan, dtype=t)
        # the codes of values above zero are the positive bytes
        grad_hidden.masked_fill_(s.hidden.values.view(torch.int8)[:, :self.hidden] <= 0, 0)
        grads["up"] = binding.gs_expert_weight_grad(s.tokens, grad_hidden, s.plan, gather=True)
        grad_sent = binding.gs_expert_product(binding.gs_quantize(grad_hidden), s.weights.up_back, s.plan, dtype=t)
        grad_logits = binding.gs_expert_route_bwd(s.logits, s.route, combine.weights, self._grad_loss)
        again = binding.gs_layer_norm_fwd(s.x, p["norm_weight"], p["norm_bias"], stats=False)
        grads["router"] = again.y.float().t() @ grad_logits
        grad_norm = binding.gs_expert_combine(grad_sent, s.plan).float() + grad_logits @ p["router"].t()
        norm = binding.gs_layer_norm_bwd(s.x, p["norm_weight"], s.mean, s.rstd, grad_norm.to(t))
        grads["norm_weight"], grads["norm_bias"] = norm.weight, norm.bias
        return grad_y + norm.x, grads

    def forward(self, x, weights=None):
        """(y, what the backward needs) of x [tokens, dim] of the layer's type. Library products: synchronises once, for
        the experts' row counts. 8-bit products: weights as hold_weights gave them (None: held for this call)."""
        if x.dtype != self.dtype:
            raise TypeError(f"x must be {self.dtype}, the layer's type (got {x.dtype})")
        if self.products == "f8":
            return self._forward_held(x, weights)
        if weights is not None:
            raise ValueError('weights go with products="f8"')
        p, T, K = self.parameters, x.shape[0], self.choices
        norm = binding.gs_layer_norm_fwd(x, p["norm_weight"], p["norm_bias"])
        logits, route = norm.y.float() @ p["router"], None
        if self.balance:
            route = binding.gs_expert_route(logits, K)
            ids, weights = route.ids, route.weights
        else:
            best, ids = logits.topk(K, dim=1)
            ids, weights = ids.to(torch.int32), best.softmax(dim=1)
        plan = binding.gs_expert_plan(ids, self.experts)
        sent = binding.gs_expert_dispatch(norm.y, plan)
        bounds = plan.offsets.tolist()
        hidden = self._of_experts(sent, p["up"].to(x.dtype), bounds, x.new_empty(T * K, self.hidden)).relu_()
        rows = self._of_experts(hidden, p["down"].to(x.dtype), bounds, torch.empty_like(sent))
        y = x + binding.gs_expert_combine(rows, plan, weights)
        return y, _Saved(x, norm, plan, bounds, ids, weights, sent, hidden, rows, None if route is None else logits, route)

    def backward(self, s, grad_y):
        """(gradient of x, gradients of the parameters by name) of sum(grad_y * y) + balance * balance loss."""
        if self.products == "f8":
            return self._backward_held(s, grad_y)
        p, t = self.parameters, s.x.dtype
        combine = binding.gs_expert_combine_bwd(s.rows, s.plan, s.weights, grad_y)
        turned = lambda w: w.to(t).transpose(1, 2).contiguous()  # noqa: E731
        grad_hidden = self._of_experts(combine.rows, turned(p["down"]), s.bounds, torch.empty_like(s.hidden))
        grad_hidden.masked_fill_(s.hidden <= 0, 0)
        grad_sent = self._of_experts(grad_hidden, turned(p["up"]), s.bounds, torch.empty_like(s.sent))
        grads = {"up": torch.zeros_like(p["up"]), "down": torch.zeros_like(p["down"])}
        for e in range(self.experts):
            of = slice(s.bounds[e], s.bounds[e + 1])
            grads["up"][e] = s.sent[of].t() @ grad_hidden[of]
            grads["down"][e] = s.hidden[of].t() @ combine.rows[of]
        if s.route is not None:
            grad_logits = binding.gs_expert_route_bwd(s.logits, s.route, combine.weights, self._grad_loss)
        else:  # the softmax over a token's chosen logits
            g = s.weights * (combine.weights - (s.weights * combine.weights).sum(dim=1, keepdim=True))
            grad_logits = torch.zeros(s.x.shape[0], self.experts, device=g.device).scatter_(1, s.ids.long(), g)
        grads["router"] = s.norm.y.float().t() @ grad_logits
        grad_norm = binding.gs_expert_combine(grad_sent, s.plan).float() + grad_logits @ p["router"].t()
        norm = binding.gs_layer_norm_bwd(s.x, p["norm_weight"], s.norm.mean, s.norm.rstd, grad_norm.to(t))
        grads["norm_weight"], grads["norm_bias"] = norm.weight, norm.bias
        return grad_y + norm.x, grads


class ColorHead(_Momentum):
    """colours = 1 / (1 + exp(-(x weight + bias)))."""

    def __init__(self, dim, channels=3, seed=1, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        super().__init__({"weight": _normal(g, dim, channels, std=dim ** -0.5),
                          "bias": torch.zeros(channels, device=device)})

    def forward(self, x):
        return torch.sigmoid(x.float() @ self.parameters["weight"] + self.parameters["bias"])

    def backward(self, x, colors, grad_colors):
        g = grad_colors * colors * (1 - colors)
        return (g @ self.parameters["weight"].t()).to(x.dtype), {"weight": x.float().t() @ g, "bias": g.sum(dim=0)}
