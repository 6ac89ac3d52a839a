"""What is measured of the operators that take a splat-predicting expert layer's routing and products into the library:
the router with its balance loss and per-expert counts and its gradient, activations kept in 8 bits and restored,
products of rows sorted by expert with 8-bit weights, and the weights' gradient from activations kept in 8 bits.

``run`` computes them in plain torch operations in 32 bits (``own`` false) or through the library's entry points
(``own`` true); ``exact`` computes them from their definitions in 64 bits.

8-bit values are e4m3 with a scale 2^e for each block of 128 values along a row, e the least with max |block| <= 448 * 2^e
(within [-126, 127]; 0 for a block of zeros); rows are padded to whole blocks with zeros.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 128
E4M3_MAX = 448.0


def listed():
    return [
        # a handful of tokens at inference: latency
        {"name": "route_fwd_few", "op": "route_fwd", "tokens": 16, "choices": 2, "experts": 8, "dtype": "f32",
         "masked": 0.0, "renormalize": True},
        # one token a splat of a scene of a million
        {"name": "route_fwd_splats", "op": "route_fwd", "tokens": 1000000, "choices": 2, "experts": 8, "dtype": "f32",
         "masked": 0.05, "renormalize": True},
        # a training batch over many small experts, eight choices each, and an odd one of 16-bit logits
        {"name": "route_bwd_train", "op": "route_bwd", "tokens": 32768, "choices": 8, "experts": 64, "dtype": "f32",
         "masked": 0.0, "renormalize": True},
        {"name": "route_bwd_odd", "op": "route_bwd", "tokens": 4999, "choices": 3, "experts": 60, "dtype": "bf16",
         "masked": 0.1, "renormalize": False},
        # a batch's activations kept from the forward and restored in the backward, and an odd width in 32 bits
        {"name": "checkpoint_train", "op": "checkpoint", "rows": 65536, "dim": 4096, "dtype": "bf16"},
        {"name": "checkpoint_odd", "op": "checkpoint", "rows": 2049, "dim": 1001, "dtype": "f32"},
        # few tokens over few experts at inference: the weights are what is read
        {"name": "product_few", "op": "product", "tokens": 16, "choices": 2, "experts": 8, "dim": 1024, "out": 2048,
         "dtype": "bf16", "dropped": 0.0, "gather": True, "relu": True},
        # many experts with some tens of rows each, odd widths, results in 32 bits
        {"name": "product_odd", "op": "product", "tokens": 1501, "choices": 3, "experts": 60, "dim": 769, "out": 1001,
         "dtype": "f32", "dropped": 0.1, "gather": False, "relu": False},
        # a training batch of a two-choice layer of large experts
        {"name": "product_train", "op": "product", "tokens": 16384, "choices": 2, "experts": 16, "dim": 4096,
         "out": 4096, "dtype": "bf16", "dropped": 0.05, "gather": True, "relu": True},
        # one token a splat of a scene of 200 thousand: small matrices, long sums
        {"name": "weight_grad_splats", "op": "weight_grad", "tokens": 200000, "choices": 2, "experts": 8, "dim": 128,
         "out": 256, "dtype": "bf16", "dropped": 0.0, "gather": True},
        # the odd layer's gradients in 32 bits, and the large layer's
        {"name": "weight_grad_odd", "op": "weight_grad", "tokens": 1501, "choices": 3, "experts": 60, "dim": 769,
         "out": 257, "dtype": "f32", "dropped": 0.1, "gather": False},
        {"name": "weight_grad_train", "op": "weight_grad", "tokens": 16384, "choices": 2, "experts": 16, "dim": 4096,
         "out": 4096, "dtype": "bf16", "dropped": 0.05, "gather": True},
    ]


def _between(rng, low, high):
    """A whole number of [low, high], spread over its logarithm; every third one odd."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return min(high, max(low, v | 1 if rng.random() < 0.34 else v))


def draw(rng):
    op = rng.choice(["route_fwd", "route_bwd", "checkpoint", "product", "weight_grad"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "checkpoint":
        dim = _between(rng, 64, 8192)
        return {"op": op, "rows": _between(rng, 1, max(1, min(1 << 20, (1 << 27) // dim))), "dim": dim, "dtype": dtype}
    experts = _between(rng, 2, 256)
    choices = rng.randint(1, min(8, experts))
    if op in ("route_fwd", "route_bwd"):
        tokens = _between(rng, 1, max(1, min(1 << 20, (1 << 25) // experts)))
        return {"op": op, "tokens": tokens, "choices": choices, "experts": experts, "dtype": dtype,
                "masked": rng.choice([0.0, 0.0, 0.1]), "renormalize": rng.choice([True, False])}
    dim, out = _between(rng, 64, 4096), _between(rng, 64, 4096)
    experts = max(choices, min(experts, (1 << 28) // (dim * out)))
    tokens = _between(rng, 1, max(1, min(200000, (1 << 38) // (dim * out * choices),
                                         (1 << 27) // (max(dim, out) * choices))))
    case = {"op": op, "tokens": tokens, "choices": choices, "experts": experts, "dim": dim, "out": out, "dtype": dtype,
            "dropped": rng.choice([0.0, 0.0, 0.1]), "gather": rng.choice([True, False])}
    if op == "product":
        case["relu"] = rng.choice([True, False])
    return case


def _normal(g, *shape, std=1.0, mean=0.0):
    return torch.randn(*shape, generator=g, device="cuda") * std + mean


def _logits(case, g):
    """A router's logits: some experts favoured."""
    T, E = case["tokens"], case["experts"]
    return _normal(g, T, E) + _normal(g, E, std=0.5)


def _channels(g, rows, dim):
    """Activations: channels of widths of their own."""
    return _normal(g, rows, dim) * torch.exp(_normal(g, dim, std=0.5))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] in ("route_fwd", "route_bwd"):
        s["logits"] = _logits(case, g).to(dt)
        s["mask"] = None
        if case["masked"]:
            s["mask"] = torch.rand(case["tokens"], generator=g, device="cuda") >= case["masked"]
        if case["op"] == "route_bwd":
            s["route"] = _plain_route(s["logits"], s["mask"], case["choices"], case["renormalize"])  # of the forward
            s["grad_weights"] = _normal(g, case["tokens"], case["choices"], std=0.1)
            s["grad_loss"] = torch.full((), 0.01, device="cuda")
        return s
    if case["op"] == "checkpoint":
        s["x"] = _channels(g, case["rows"], case["dim"]).to(dt)
        return s
    T, K, E, D, N = case["tokens"], case["choices"], case["experts"], case["dim"], case["out"]
    ids = torch.sort(_logits(case, g), dim=1, descending=True, stable=True).indices[:, :K].to(torch.int32)
    if case["dropped"]:
        ids = torch.where(torch.rand(T, K, generator=g, device="cuda") < case["dropped"], -1, ids)
    s["offsets"], s["rows"], s["pairs"] = _plain_plan(ids.contiguous(), E)
    s["x"] = _plain_quantize(_channels(g, T if case["gather"] else T * K, D))
    if case["op"] == "product":
        s["weight"] = _plain_quantize(_normal(g, E, N, D, std=D ** -0.5))
    else:
        s["grad"] = (_normal(g, T * K, N, std=0.1) * (s["pairs"] >= 0)[:, None]).to(dt)
    return s


def _plain_plan(ids, experts):
    flat = ids.reshape(-1)
    valid = (flat >= 0) & (flat < experts)
    key = torch.where(valid, flat, experts).long()
    ordered, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ordered, torch.arange(experts + 1, device=flat.device))
    place = torch.empty_like(order)
    place[order] = torch.arange(flat.numel(), device=flat.device)
    rows = torch.where(valid, place, -1).reshape(ids.shape)
    pairs = torch.where(valid[order], order, -1)
    return offsets.to(torch.int32), rows.to(torch.int32), pairs.to(torch.int32)


def _power32(e):
    """2^e for whole numbers e of [-126, 127]."""
    return (e + 127 << 23).to(torch.int32).view(torch.float32)


def _plain_quantize(x):
    """(e4m3 values [..., blocks * 128], scale bytes [..., blocks]) of the rows of x."""
    dim = x.shape[-1]
    blocks = -(-dim // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - dim)).unflatten(-1, (blocks, BLOCK))
    m, e = torch.frexp(v.abs().amax(dim=-1))  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m == 0, 0, torch.where(m > 0.875, e - 8, e - 9).clamp(-126, 127))
    values = (v * _power32(-e)[..., None]).to(torch.float8_e4m3fn)
    return values.flatten(-2), (e + 127).to(torch.uint8)


def _plain_dequantize(q, dim):
    values, scales = q
    v = values.float().unflatten(-1, (-1, BLOCK))
    return (v * _power32(scales.int() - 127)[..., None]).flatten(-2)[..., :dim]


def _plain_route(logits, mask, choices, renormalize):
    """(ids, weights, counts, shares, loss, kept)."""
    T, E = logits.shape
    x = logits.float()
    e = torch.exp(x - x.amax(dim=1, keepdim=True))
    p = e / e.sum(dim=1, keepdim=True)
    best, ids = (a[:, :choices] for a in torch.sort(x, dim=1, descending=True, stable=True))
    if renormalize:
        weights = torch.exp(best - best[:, :1])
        weights = weights / weights.sum(dim=1, keepdim=True)
    else:
        weights = p.gather(1, ids)
    ids = ids.to(torch.int32)
    kept = torch.ones(T, dtype=torch.bool, device=x.device) if mask is None else mask
    ids, weights = torch.where(kept[:, None], ids, -1), torch.where(kept[:, None], weights, 0.0)
    n = kept.sum()
    counts = torch.zeros(E + 1, dtype=torch.int32, device=x.device)
    counts = counts.index_add(0, ids.reshape(-1) + 1, torch.ones_like(ids).reshape(-1))[1:]
    shares = torch.where(kept[:, None], p, 0.0).sum(dim=0) / n.clamp(min=1)
    loss = E * (counts / counts.sum().clamp(min=1) * shares).sum()
    return ids, weights, counts, shares, loss, n.to(torch.int32).reshape(1)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    dt = DTYPES[case["dtype"]]
    if op == "route_fwd":
        ids, weights, counts, shares, loss, _ = _plain_route(s["logits"], s["mask"], case["choices"],
                                                             case["renormalize"])
        return {"ids": ids, "weights": weights, "counts": counts, "shares": shares, "loss": loss}
    if op == "route_bwd":
        ids, weights, counts, _, _, n = s["route"]
        x = s["logits"].float()
        e = torch.exp(x - x.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
        kept, at = (ids >= 0), ids.clamp(min=0).long()
        g = torch.where(kept, s["grad_weights"] * weights, 0.0)  # of the chosen logits, before the normalisation's part
        total = g.sum(dim=1, keepdim=True)
        f = counts / counts.sum().clamp(min=1)
        balance = p * (f - (p * f).sum(dim=1, keepdim=True)) * (s["grad_loss"] * x.shape[1] / n.clamp(min=1))
        if case["renormalize"]:
            gx = balance.scatter_add(1, at, g - torch.where(kept, weights, 0.0) * total)
        else:
            gx = (balance - p * total).scatter_add(1, at, g)
        return torch.where(kept[:, :1], gx, 0.0).to(dt)
    if op == "checkpoint":
        largest = torch.finfo(dt).max
        return _plain_dequantize(_plain_quantize(s["x"]), case["dim"]).clamp(-largest, largest).to(dt)
    K, D, N = case["choices"], case["dim"], case["out"]
    bounds = s["offsets"].tolist()
    x = _plain_dequantize(s["x"], D)
    if case["gather"]:
        x = x[(s["pairs"].clamp(min=0) // K).long()]
    if op == "product":
        w = _plain_dequantize(s["weight"], D)
        out = torch.zeros(x.shape[0], N, device=x.device)
        for e in range(case["experts"]):
            of = slice(bounds[e], bounds[e + 1])
            out[of] = torch.matmul(x[of], w[e].t())
        return (out.clamp(min=0) if case["relu"] else out).to(dt)
    out = torch.zeros(case["experts"], D, N, device=x.device)
    for e in range(case["experts"]):
        of = slice(bounds[e], bounds[e + 1])
        out[e] = torch.matmul(x[of].t(), s["grad"][of].float())
    return out


def _own(s):
    from tile_binned_gaussian_amd import binding as gs
    case, op = s["case"], s["case"]["op"]
    dt = DTYPES[case["dtype"]]
    if op == "route_fwd":
        r = gs.gs_expert_route(s["logits"], case["choices"], mask=s["mask"], renormalize=case["renormalize"])
        return {"ids": r.ids, "weights": r.weights, "counts": r.counts, "shares": r.shares, "loss": r.loss}
    if op == "route_bwd":
        return gs.gs_expert_route_bwd(s["logits"], gs.ExpertRoute(*s["route"]), s["grad_weights"], s["grad_loss"],
                                      renormalize=case["renormalize"])
    if op == "checkpoint":
        return gs.gs_dequantize(gs.gs_quantize(s["x"]), dtype=dt)
    plan = gs.ExpertPlan(s["offsets"], s["rows"], s["pairs"])
    x = gs.Quantized(*s["x"], case["dim"])
    if op == "product":
        return gs.gs_expert_product(x, gs.Quantized(*s["weight"], case["dim"]), plan, gather=case["gather"],
                                       relu=case["relu"], dtype=dt)
    return gs.gs_expert_weight_grad(x, s["grad"], plan, gather=case["gather"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, es = case["op"], BYTES[case["dtype"]]
    if op == "checkpoint":
        R, D = case["rows"], case["dim"]
        held = R * -(-D // BLOCK) * (BLOCK + 1)
        return {"bytes": 2 * R * D * es + 2 * held, "flops": 4 * R * D}
    T, K, E = case["tokens"], case["choices"], case["experts"]
    if op == "route_fwd":
        return {"bytes": T * E * es + 8 * T * K + 8 * E + (T if case["masked"] else 0), "flops": 5 * T * E}
    if op == "route_bwd":
        return {"bytes": 2 * T * E * es + 12 * T * K + 4 * E, "flops": 9 * T * E}
    D, N = case["dim"], case["out"]
    held = -(-D // BLOCK) * (BLOCK + 1)
    kept = int(T * K * (1.0 - case["dropped"]))
    used = min(E, max(1, kept))
    rows = (min(T, kept) if case["gather"] else kept) * held
    if op == "product":
        return {"bytes": rows + used * N * held + T * K * N * es + 4 * T * K, "flops": 2 * kept * D * N}
    return {"bytes": rows + kept * N * es + 4 * E * D * N + 4 * T * K, "flops": 2 * kept * D * N}


def _power64(e):
    """2^e for whole numbers e of [-300, 300]."""
    table = torch.tensor([2.0 ** k for k in range(-300, 301)], dtype=torch.float64, device=e.device)
    return table[e.long() + 300]


def _values64(q, dim):
    """What 8-bit rows stand for, scale by scale."""
    values, scales = q
    step = _power64(scales.long() - 127).repeat_interleave(BLOCK, dim=-1)
    return (values.double() * step)[..., :dim]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("route_fwd", "route_bwd"):
        T, E, K = case["tokens"], case["experts"], case["choices"]
        x = s["logits"].double().requires_grad_(op == "route_bwd")
        kept = torch.arange(T, device="cuda") if s["mask"] is None else torch.nonzero(s["mask"])[:, 0]
        # the K largest, the lower index first among equal ones
        order = torch.argsort(-x.detach()[kept], dim=1, stable=True)[:, :K]
        p = torch.softmax(x[kept], dim=1)
        chosen = x[kept].gather(1, order)
        w = torch.softmax(chosen, dim=1) if case["renormalize"] else p.gather(1, order)
        counts = torch.bincount(order.reshape(-1), minlength=E).double()
        n = max(1, kept.numel())
        shares = p.sum(dim=0) / n
        loss = E * torch.dot(counts / max(1, kept.numel() * K), shares)
        if op == "route_fwd":
            weights = torch.zeros(T, K, dtype=torch.float64, device="cuda")
            weights[kept] = w
            return {"ids": None, "weights": weights, "counts": None, "shares": shares, "loss": loss}
        # the forward's weights are stored in 32 bits, and its gradient is taken at them: no more than 2^-24 apart
        total = (w * s["grad_weights"][kept].double()).sum() + loss * s["grad_loss"].double()
        return torch.autograd.grad(total, x)[0]
    if op == "checkpoint":
        # by steps of the grid around each value: 2^-3 of its power of two, not below the scale's 2^-9; ties to even
        x, dim = s["x"].double(), case["dim"]
        out = torch.empty_like(x)
        for at in range(0, dim, BLOCK):
            b = x[:, at:at + BLOCK]
            most = b.abs().amax(dim=1, keepdim=True)
            e = torch.ceil(torch.log2(torch.where(most > 0, most, 448.0) / 448.0) - 1e-12).clamp(-126, 127)
            e = torch.where(most > 448.0 * _power64(e), e + 1, e)
            power = torch.floor(torch.log2(torch.where(b == 0, 1.0, b.abs())))
            power = torch.where(_power64(power) > b.abs(), power - 1, power)
            power = torch.where(_power64(power + 1) <= b.abs(), power + 1, power)
            step = torch.maximum(_power64(power - 3), _power64(e - 9))
            out[:, at:at + BLOCK] = torch.round(b / step) * step
        largest = torch.finfo(DTYPES[case["dtype"]]).max
        return out.clamp(-largest, largest)
    K, D, N, E = case["choices"], case["dim"], case["out"], case["experts"]
    if 2.0 * case["tokens"] * K * D * N > 4e12:
        return None
    bounds = s["offsets"].tolist()
    x = _values64(s["x"], D)
    source = s["pairs"].long() // K if case["gather"] else torch.arange(case["tokens"] * K, device="cuda")
    out = torch.zeros((case["tokens"] * K, N) if op == "product" else (E, D, N), dtype=torch.float64, device="cuda")
    for e in range(E):
        of = slice(bounds[e], bounds[e + 1])
        if bounds[e] == bounds[e + 1]:
            continue
        rows = x[source[of]]
        if op == "product":
            w = _values64((s["weight"][0][e], s["weight"][1][e]), D)
            out[of] = torch.mm(rows, w.t().contiguous())
        else:
            torch.mm(rows.t().contiguous(), s["grad"][of].double(), out=out[e])
    return torch.relu_(out) if op == "product" and case["relu"] else out
