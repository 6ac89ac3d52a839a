"""What is measured of the training operators around a splat-predicting expert layer: layer norm and its gradient,
tokens sorted by expert and back and its gradient, and the orthogonalised update of a weight matrix.

``run`` computes them in plain torch operations in 32 bits (``own`` false) or through the library's entry points
(``own`` true); ``exact`` computes them from their definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5  # layer norm
STEPS = 5  # orthogonalisation: steps, coefficients of X, A X and A A X, and the norm's guard
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
NORM_EPS = 1e-7


def listed():
    return [
        # a handful of tokens at inference: latency
        {"name": "norm_fwd_few", "op": "norm_fwd", "rows": 8, "dim": 1024, "dtype": "bf16", "weight": "bf16"},
        # a training batch with weights kept in 32 bits
        {"name": "norm_fwd_train", "op": "norm_fwd", "rows": 32768, "dim": 2048, "dtype": "bf16", "weight": "f32"},
        # an odd width, rows that start at every alignment
        {"name": "norm_fwd_odd", "op": "norm_fwd", "rows": 4999, "dim": 1537, "dtype": "f32", "weight": "f32"},
        # the same layer's backward, a wide one and an odd one
        {"name": "norm_bwd_train", "op": "norm_bwd", "rows": 32768, "dim": 4096, "dtype": "bf16", "weight": "f32"},
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 2049, "dim": 1001, "dtype": "f16", "weight": "f32"},
        # few tokens over few experts at inference: latency
        {"name": "experts_fwd_few", "op": "experts_fwd", "tokens": 16, "choices": 2, "experts": 8, "dim": 1024,
         "dtype": "bf16", "dropped": 0.0},
        # a training batch over many small experts, eight choices each
        {"name": "experts_fwd_train", "op": "experts_fwd", "tokens": 32768, "choices": 8, "experts": 64, "dim": 2048,
         "dtype": "bf16", "dropped": 0.0},
        # the backward of a two-choice layer with a capacity that drops some choices, and an odd small one
        {"name": "experts_bwd_train", "op": "experts_bwd", "tokens": 16384, "choices": 2, "experts": 16, "dim": 4096,
         "dtype": "bf16", "dropped": 0.05},
        {"name": "experts_bwd_odd", "op": "experts_bwd", "tokens": 1501, "choices": 3, "experts": 60, "dim": 769,
         "dtype": "f32", "dropped": 0.1},
        # the updates of a stack of small matrices
        {"name": "ortho_stack", "op": "ortho", "batch": 16, "m": 96, "n": 160, "dtype": "f32"},
        # a tall matrix of odd sides, momentum kept in 32 bits
        {"name": "ortho_odd", "op": "ortho", "batch": 1, "m": 2500, "n": 1111, "dtype": "f32"},
        # a large square layer, momentum in bfloat16
        {"name": "ortho_large", "op": "ortho", "batch": 1, "m": 4096, "n": 4096, "dtype": "bf16"},
    ]


def _between(rng, low, high):
    """A whole number of [low, high], spread over its logarithm; every third one odd."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return min(high, max(low, v | 1 if rng.random() < 0.34 else v))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "experts_fwd", "experts_bwd", "ortho"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("norm_fwd", "norm_bwd"):
        dim = _between(rng, 64, 8192)
        rows = _between(rng, 1, max(1, min(65536, (1 << 26) // dim)))
        return {"op": op, "rows": rows, "dim": dim, "dtype": dtype, "weight": rng.choice(["f32", dtype])}
    if op in ("experts_fwd", "experts_bwd"):
        experts = _between(rng, 2, 256)
        choices = rng.randint(1, min(8, experts))
        dim = _between(rng, 64, 4096)
        tokens = _between(rng, 1, max(1, min(32768, (1 << 27) // (dim * choices))))
        return {"op": op, "tokens": tokens, "choices": choices, "experts": experts, "dim": dim, "dtype": dtype,
                "dropped": rng.choice([0.0, 0.0, 0.1])}
    m, n = _between(rng, 32, 4096), _between(rng, 32, 4096)
    batch = max(1, min(_between(rng, 1, 16), int(4096 ** 3 / 8 / (min(m, n) ** 2 * max(m, n)))))
    return {"op": op, "batch": batch, "m": m, "n": n, "dtype": dtype}


def _normal(g, *shape, std=1.0, mean=0.0):
    return torch.randn(*shape, generator=g, device="cuda") * std + mean


def _plan_inputs(case, g):
    """A router's choices: the best `choices` of uneven logits, their softmax weights, some choices dropped (-1)."""
    T, K, E = case["tokens"], case["choices"], case["experts"]
    logits = _normal(g, T, E) + _normal(g, E, std=0.5)
    best, ids = logits.topk(K, dim=1)
    ids = ids.to(torch.int32)
    if case["dropped"]:
        ids = torch.where(torch.rand(T, K, generator=g, device="cuda") < case["dropped"], -1, ids)
    return ids.contiguous(), best.softmax(dim=1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] in ("norm_fwd", "norm_bwd"):
        R, D, wt = case["rows"], case["dim"], DTYPES[case["weight"]]
        # channels with offsets and widths of their own, as residual streams have
        x = _normal(g, R, D) * torch.exp(_normal(g, D, std=0.5)) + _normal(g, D, std=0.5)
        s["x"] = x.to(dt)
        s["weight"] = _normal(g, D, std=0.1, mean=1.0).to(wt)
        s["bias"] = _normal(g, D, std=0.1).to(wt)
        if case["op"] == "norm_bwd":
            s["grad_y"] = _normal(g, R, D, std=0.1).to(dt)
            xd = s["x"].float()
            s["mean"] = xd.mean(dim=1)
            s["rstd"] = torch.rsqrt((xd - s["mean"][:, None]).square().mean(dim=1) + EPS)
        return s
    if case["op"] in ("experts_fwd", "experts_bwd"):
        T, K, D = case["tokens"], case["choices"], case["dim"]
        s["ids"], s["weights"] = _plan_inputs(case, g)
        s["expert_rows"] = _normal(g, T * K, D).to(dt)  # what the experts gave for the sorted rows
        if case["op"] == "experts_fwd":
            s["x"] = _normal(g, T, D).to(dt)
        else:
            s["offsets"], s["rows"], s["pairs"] = _plain_plan(s["ids"], case["experts"])  # kept from the forward
            s["grad_y"] = _normal(g, T, D, std=0.1).to(dt)
            s["grad_rows"] = _normal(g, T * K, D, std=0.1).to(dt)  # gradient at the dispatched rows
        return s
    B, m, n = case["batch"], case["m"], case["n"]
    r = max(1, min(m, n) // 32)  # momentum: a few strong directions and a bulk of weak ones
    left, right = _normal(g, B, m, r), _normal(g, B, r, n)
    s["update"] = (torch.matmul(left, right) * (1e-3 / r ** 0.5) + _normal(g, B, m, n, std=3e-4)).to(dt)
    return s


def _plain_plan(ids, experts):
    flat = ids.reshape(-1)
    valid = (flat >= 0) & (flat < experts)
    key = torch.where(valid, flat, experts).long()
    ordered, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ordered, torch.arange(experts + 1, device=flat.device))
    at = torch.arange(flat.numel(), device=flat.device)
    place = torch.empty_like(at)
    place[order] = at
    rows = torch.where(valid, place, -1).reshape(ids.shape)
    pairs = torch.where(valid[order], order, -1)
    return offsets.to(torch.int32), rows.to(torch.int32), pairs.to(torch.int32)


def _plain_combine(source, rows, weights):
    """sum over a token's kept choices of weight times row, in 32 bits."""
    kept = rows >= 0
    picked = torch.where(kept[:, :, None], source[rows.clamp(min=0).long()].float(), 0.0)
    return (picked if weights is None else picked * weights[:, :, None]).sum(dim=1)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    dt = DTYPES[case["dtype"]]
    if op == "norm_fwd":
        x = s["x"].float()
        mean = x.mean(dim=1, keepdim=True)
        c = x - mean
        rstd = torch.rsqrt(c.square().mean(dim=1, keepdim=True) + EPS)
        y = c * rstd * s["weight"].float() + s["bias"].float()
        return {"y": y.to(dt), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if op == "norm_bwd":
        x, gy, rstd = s["x"].float(), s["grad_y"].float(), s["rstd"][:, None]
        xh = (x - s["mean"][:, None]) * rstd
        g = gy * s["weight"].float()
        gx = rstd * (g - g.mean(dim=1, keepdim=True) - xh * (g * xh).mean(dim=1, keepdim=True))
        wt = s["weight"].dtype
        return {"grad_x": gx.to(dt), "grad_weight": (gy * xh).sum(dim=0).to(wt), "grad_bias": gy.sum(dim=0).to(wt)}
    if op == "experts_fwd":
        offsets, rows, pairs = _plain_plan(s["ids"], case["experts"])
        sent = torch.where((pairs >= 0)[:, None], s["x"][(pairs.clamp(min=0) // case["choices"]).long()], 0)
        y = _plain_combine(s["expert_rows"], rows, s["weights"]).to(dt)
        return {"offsets": offsets, "rows": rows, "pairs": pairs, "sent": sent, "y": y}
    if op == "experts_bwd":
        rows, pairs, K = s["rows"], s["pairs"], case["choices"]
        kept = (pairs >= 0)[:, None]
        at = pairs.clamp(min=0).long()
        gy = s["grad_y"].float()[at // K]
        grad_in = torch.where(kept, gy * s["weights"].reshape(-1)[at][:, None], 0.0).to(dt)
        dots = torch.where(kept[:, 0], (gy * s["expert_rows"].float()).sum(dim=1), 0.0)
        grad_w = torch.where(rows >= 0, dots[rows.clamp(min=0).long()], 0.0)
        return {"grad_expert_rows": grad_in, "grad_weights": grad_w,
                "grad_x": _plain_combine(s["grad_rows"], rows, None).to(dt)}
    a, b, c = COEFFICIENTS
    x = s["update"].float()
    tall = case["m"] > case["n"]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + NORM_EPS)
    for _ in range(STEPS):
        A = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * A + c * torch.matmul(A, A), x)
    return (x.transpose(1, 2) if tall else x).to(dt).contiguous()


def _own(s):
    from tile_binned_gaussian_amd import binding as gs
    case, op = s["case"], s["case"]["op"]
    if op == "norm_fwd":
        r = gs.gs_layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=EPS)
        return {"y": r.y, "mean": r.mean, "rstd": r.rstd}
    if op == "norm_bwd":
        r = gs.gs_layer_norm_bwd(s["x"], s["weight"], s["mean"], s["rstd"], s["grad_y"])
        return {"grad_x": r.x, "grad_weight": r.weight, "grad_bias": r.bias}
    if op == "experts_fwd":
        plan = gs.gs_expert_plan(s["ids"], case["experts"])
        sent = gs.gs_expert_dispatch(s["x"], plan)
        y = gs.gs_expert_combine(s["expert_rows"], plan, s["weights"])
        return {"offsets": plan.offsets, "rows": plan.rows, "pairs": plan.pairs, "sent": sent, "y": y}
    if op == "experts_bwd":
        plan = gs.ExpertPlan(s["offsets"], s["rows"], s["pairs"])
        r = gs.gs_expert_combine_bwd(s["expert_rows"], plan, s["weights"], s["grad_y"])
        return {"grad_expert_rows": r.rows, "grad_weights": r.weights,
                "grad_x": gs.gs_expert_combine(s["grad_rows"], plan)}
    return gs.gs_orthogonalize(s["update"], steps=STEPS, coefficients=COEFFICIENTS, eps=NORM_EPS)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, es = case["op"], BYTES[case["dtype"]]
    if op in ("norm_fwd", "norm_bwd"):
        R, D, ws = case["rows"], case["dim"], BYTES[case["weight"]]
        if op == "norm_fwd":
            return {"bytes": 2 * R * D * es + 8 * R + 2 * D * ws, "flops": 8 * R * D}
        return {"bytes": 3 * R * D * es + 8 * R + 3 * D * ws, "flops": 14 * R * D}
    if op in ("experts_fwd", "experts_bwd"):
        T, K, D, E = case["tokens"], case["choices"], case["dim"], case["experts"]
        kept = T * K * (1.0 - case["dropped"])
        if op == "experts_fwd":  # ids and plan; x once, the sorted rows, the experts' rows, y
            return {"bytes": int(12 * T * K + 4 * E + (T + T * K) * D * es + (kept + T) * D * es + 4 * T * K),
                    "flops": int(2 * kept * D)}
        return {"bytes": int(4 * T * K + (T + kept + T * K) * D * es + 8 * T * K + (kept + T) * D * es),
                "flops": int(4 * kept * D)}
    M, N, B = min(case["m"], case["n"]), max(case["m"], case["n"]), case["batch"]
    # the two symmetric products need half of their entries
    return {"bytes": 2 * B * M * N * es, "flops": STEPS * B * (3 * M * M * N + M * M * M)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
        y = (x - mean) / (var + EPS).sqrt() * s["weight"].double() + s["bias"].double()
        return {"y": y, "mean": mean[:, 0], "rstd": (var + EPS).pow(-0.5)[:, 0]}
    if op == "norm_bwd":  # by the chain rule through the centred row; the statistics are the given ones
        x, w = s["x"].double(), s["weight"].double()
        gy, mean, rstd = s["grad_y"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
        D = case["dim"]
        scaled = gy * w * rstd
        pull = (scaled * (x - mean)).sum(dim=1, keepdim=True) * rstd.square() / D
        gx = scaled - (x - mean) * pull - scaled.sum(dim=1, keepdim=True) / D
        return {"grad_x": gx, "grad_weight": torch.einsum("rd,rd->d", gy, (x - mean) * rstd),
                "grad_bias": gy.sum(dim=0)}
    if op in ("experts_fwd", "experts_bwd"):
        T, K, D = case["tokens"], case["choices"], case["dim"]
        flat = s["ids"].reshape(-1)
        keep = torch.nonzero((flat >= 0) & (flat < case["experts"]))[:, 0]
        # sorted by (expert, choice): the pair's own number breaks ties
        order = keep[torch.argsort(flat[keep].long() * (T * K) + keep)]
        token, w, n = order // K, s["weights"].reshape(-1)[order].double()[:, None], order.numel()
        if op == "experts_fwd":
            sent = torch.zeros(T * K, D, dtype=torch.float64, device="cuda")
            sent[:n] = s["x"][token].double()
            y = torch.zeros(T, D, dtype=torch.float64, device="cuda")
            y.index_add_(0, token, s["expert_rows"][:n].double() * w)
            return {"offsets": None, "rows": None, "pairs": None, "sent": sent, "y": y}
        gy = s["grad_y"].double()
        grad_in = torch.zeros(T * K, D, dtype=torch.float64, device="cuda")
        grad_in[:n] = gy[token] * w
        grad_w = torch.zeros(T * K, dtype=torch.float64, device="cuda")
        grad_w[order] = (gy[token] * s["expert_rows"][:n].double()).sum(dim=1)
        grad_x = torch.zeros(T, D, dtype=torch.float64, device="cuda")
        grad_x.index_add_(0, token, s["grad_rows"][:n].double())
        return {"grad_expert_rows": grad_in, "grad_weights": grad_w.reshape(T, K), "grad_x": grad_x}
    # the odd polynomial applied through the smaller Gram matrix, factor by factor
    a, b, c = COEFFICIENTS
    x = s["update"].double()
    x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + NORM_EPS)
    wide = case["m"] <= case["n"]
    for _ in range(STEPS):
        xt = x.transpose(1, 2).contiguous()
        if wide:
            gram = torch.bmm(x, xt)
            x = a * x + torch.bmm(gram, b * x + c * torch.bmm(gram, x))
        else:
            gram = torch.bmm(xt, x)
            x = a * x + torch.bmm(b * x + c * torch.bmm(x, gram), gram)
    return x
