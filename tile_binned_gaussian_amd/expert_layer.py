"""A layer of experts over splat features, trained through the library's entry points.

``ExpertLayer`` is a residual layer, y = x + experts(layer norm(x)): a router picks each token's best experts, the
tokens are sorted by expert, every expert is a two-layer perceptron on its own rows, and the weighted results return
to their tokens. The backward is written out call by call; weight matrices move by their orthogonalised momentum.
The experts' own products are plain library products, one per expert and direction. ``ColorHead`` maps features to
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


class ExpertLayer(_Momentum):
    def __init__(self, dim, hidden, experts, choices, seed=0, device="cuda", dtype=torch.bfloat16):
        g = torch.Generator(device=device).manual_seed(seed)
        self.experts, self.choices, self.dtype, self.hidden = experts, choices, dtype, hidden
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

    def forward(self, x):
        """(y, what the backward needs) of x [tokens, dim] of the layer's type. Synchronises once, for the experts' row
        counts."""
        if x.dtype != self.dtype:
            raise TypeError(f"x must be {self.dtype}, the layer's type (got {x.dtype})")
        p, T, K = self.parameters, x.shape[0], self.choices
        norm = binding.gs_layer_norm_fwd(x, p["norm_weight"], p["norm_bias"])
        best, ids = (norm.y.float() @ p["router"]).topk(K, dim=1)
        ids, weights = ids.to(torch.int32), best.softmax(dim=1)
        plan = binding.gs_expert_plan(ids, self.experts)
        sent = binding.gs_expert_dispatch(norm.y, plan)
        bounds = plan.offsets.tolist()
        hidden = self._of_experts(sent, p["up"].to(x.dtype), bounds, x.new_empty(T * K, self.hidden)).relu_()
        rows = self._of_experts(hidden, p["down"].to(x.dtype), bounds, torch.empty_like(sent))
        y = x + binding.gs_expert_combine(rows, plan, weights)
        return y, _Saved(x, norm, plan, bounds, ids, weights, sent, hidden, rows)

    def backward(self, s, grad_y):
        """(gradient of x, gradients of the parameters by name) of sum(grad_y * y)."""
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
        # the softmax over a token's chosen logits
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
