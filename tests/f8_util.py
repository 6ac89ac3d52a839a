"""Plain 64-bit forms of the router, of values held in 8 bits and of their products (CPU tensors), and the error bounds
that their GPU results are held to.

The bounds count roundings as train_util's do. A matrix instruction adds its products (64 of 8 bits, 16 of bfloat16), at
most one step of float32 (2^-23, cut off or rounded) for each of them, to its accumulator, one step more.
"""
import torch

from train_util import U, rounding

STEP = 2.0 ** -23


def power(e):
    """2^e of whole numbers, exact."""
    return torch.ldexp(torch.ones((), dtype=torch.float64), e.to(torch.float64))


# ----------------------------------------------------------------------------------------------------------------
# values in 8 bits


def quantize(x):
    """(values float64 as multiples of the scale, scale bytes) of the rows of x [..., dim], padded to whole blocks."""
    dim = x.shape[-1]
    blocks = -(-dim // 128)
    v = torch.nn.functional.pad(x.double(), (0, blocks * 128 - dim)).unflatten(-1, (blocks, 128))
    finite = torch.isfinite(v)
    most = torch.where(finite, v.abs(), 0.0).amax(dim=-1)
    e = torch.full_like(most, -126.0)
    for _ in range(260):  # the least that holds the block, one by one
        e = torch.where(most > 448 * power(e), e + 1, e)
    e = torch.where(most == 0, 0.0, e)
    scaled = v / power(e)[..., None]
    m, k = torch.frexp(torch.where(finite, scaled, 0.0).abs())
    step = power((k - 1).clamp(min=-6) - 3)  # three bits after the leading one; 2^-9 below the least normal, 2^-6
    q = torch.where(finite, torch.round(scaled / step) * step, float("nan"))
    return q.flatten(-2), (e + 127).to(torch.uint8)


def values_of(q, scales, dim):
    """What held values (CPU tensors, e4m3 or their float64 numbers) stand for."""
    v = q.double().unflatten(-1, (-1, 128)) * power(scales.double() - 127)[..., None]
    return v.flatten(-2)[..., :dim]


def held(q):
    """The numbers that a binding.Quantized on the GPU stands for, in 64 bits."""
    return values_of(q.values.cpu().float(), q.scales.cpu(), q.dim)


# ----------------------------------------------------------------------------------------------------------------
# the router


def choose(x, choices):
    """[T, K] experts by K passes over the row: NaN first, then the largest; -inf never; -1 where none is left."""
    ids = torch.full((x.shape[0], choices), -1, dtype=torch.int32)
    rows = x.tolist()
    for t, row in enumerate(rows):
        left = dict(enumerate(row))
        for k in range(choices):
            best = None
            for e, v in left.items():
                if v == float("-inf"):
                    continue
                if best is None or (v != v and left[best] == left[best]) or v > left[best]:
                    best = e
            if best is None:
                break
            ids[t, k] = best
            del left[best]
    return ids


def route(logits, choices, mask=None, renormalize=True, ids=None):
    """(ids, weights, counts, shares, loss, kept); differentiable in float64 logits for given ids."""
    x = logits.double()
    T, E = x.shape
    if ids is None:
        ids = choose(x.detach(), choices)
        if mask is not None:
            ids[~mask] = -1
    kept = ids[:, 0] >= 0
    chosen = ids >= 0
    p = torch.softmax(torch.where(kept[:, None], x, 0.0), dim=1)
    at = ids.clamp(min=0).long()
    if renormalize:
        picked = torch.where(chosen, x.gather(1, at), float("-inf"))
        w = torch.softmax(torch.where(kept[:, None], picked, 0.0), dim=1)
    else:
        w = p.gather(1, at)
    w = torch.where(chosen, w, 0.0)
    counts = torch.bincount(ids[chosen].long(), minlength=E)
    n = int(kept.sum())
    shares = p[kept].sum(dim=0) / max(1, n)
    loss = E * (counts.double() / max(1, int(counts.sum())) * shares).sum()
    return ids, w, counts, shares, loss, n


def spread(x):
    """Largest finite distance of a row's logits from its largest: a difference is rounded once, and exp of it is off by
    that much relative to itself."""
    x = x.double()
    d = x.amax(dim=1, keepdim=True) - x
    return torch.where(torch.isfinite(d), d, 0.0).amax(dim=1)


def route_bounds(logits, ids, w, shares, counts, kept):
    """Bounds of weights, shares and loss. A probability is two exponentials, each off by 2 steps and its argument's
    rounding, a sum of chains of at most 64 + 6 and three more operations; a share is a sum of at most 64 tokens, of
    tokens / 64 of such sums in one lane at most, and of 256 lanes."""
    T, E = logits.shape
    rel = 2 * STEP * (4 + spread(logits)) + U * 80
    most = rel.max().item() if T else 0.0
    e_shares = shares * (most + U * (64 + T / 64 / 16 + 256 + 4)) + 1e-40
    f = counts.double() / max(1, int(counts.sum()))
    return rel[:, None] * w + 1e-40, e_shares, E * (f * e_shares).sum() + 8 * U * E * (f * shares).sum() + 1e-40


def route_grad(logits, ids, weights, counts, kept, grad_weights, grad_loss, renormalize):
    """(gradient of the logits, size of its terms), at the stored weights."""
    x, w = logits.double(), weights.double()
    T, E = x.shape
    chosen, at = ids >= 0, ids.clamp(min=0).long()
    g = torch.where(chosen, grad_weights.double(), 0.0)
    routed = ids[:, :1] >= 0
    p = torch.softmax(torch.where(routed, x, 0.0), dim=1)
    total, size_total = (g * w).sum(dim=1, keepdim=True), (g * w).abs().sum(dim=1, keepdim=True)
    f = counts.double() / max(1, int(counts.sum()))
    mean = (p * f).sum(dim=1, keepdim=True)
    scale = float(grad_loss) * E / max(1, kept)
    out = p * (f - mean) * scale
    size = p * (f + mean) * abs(scale)
    if renormalize:
        out = out.scatter_add(1, at, torch.where(chosen, w * (g - total), 0.0))
        size = size.scatter_add(1, at, torch.where(chosen, w * (g.abs() + size_total), 0.0))
    else:
        out = (out - p * total).scatter_add(1, at, torch.where(chosen, w * g, 0.0))
        size = (size + p * size_total).scatter_add(1, at, torch.where(chosen, w * g.abs(), 0.0))
    return torch.where(routed, out, 0.0), torch.where(routed, size, 0.0)


def route_grad_bound(logits, grad, size, choices):
    rel = 2 * STEP * (4 + spread(logits)) + U * (100 + choices)
    return 2 * rel[:, None] * size + rounding(grad, logits.dtype) + 1e-40


# ----------------------------------------------------------------------------------------------------------------
# products


def row_experts(offsets, rows):
    """[rows] the expert of each sorted row, -1 past the kept ones."""
    of = torch.full((rows,), -1, dtype=torch.int64)
    for e in range(offsets.numel() - 1):
        of[int(offsets[e]):int(offsets[e + 1])] = e
    return of


def sorted_rows(x, pairs, choices):
    """Tokens' rows in the plan's order (row 0 where there is none)."""
    return x[(pairs.clamp(min=0) // choices).long()]


def group_most(x, w):
    """sum over groups of 8 neighbours along k of the largest |x w| of the group, [R, N]."""
    pad = -x.shape[1] % 8
    x, w = (torch.nn.functional.pad(t, (0, pad)).abs().unflatten(1, (-1, 8)) for t in (x, w))
    out = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64)
    for k in range(x.shape[1]):
        out += (x[:, None, k] * w[None, :, k]).amax(dim=-1)
    return out


def product(x, w, offsets):
    """(out, size of its terms, largest terms of groups of 8) of sorted rows x [R, D] and w [E, N, D] in 64 bits."""
    R, N = x.shape[0], w.shape[1]
    out, size, most = (torch.zeros(R, N, dtype=torch.float64) for _ in range(3))
    for e in range(w.shape[0]):
        of = slice(int(offsets[e]), int(offsets[e + 1]))
        out[of] = x[of] @ w[e].T
        size[of] = x[of].abs() @ w[e].T.abs()
        most[of] = group_most(x[of], w[e])
    return out, size, most


def product_bound(out, size, most, dim, dtype):
    """16-bit results: the 8-bit instruction cuts each of the 8 products of a group 2^-13 below the largest one's power of
    two, which is at most that product itself."""
    cut = 0.0 if dtype == torch.float32 else 7 * 2.0 ** -13 * most
    return (dim / 16 + 1 + 64) * STEP * size + cut + rounding(out, dtype)


def weight_grad(x, g, offsets):
    """(out, size of its terms) [E, D, N]."""
    E = offsets.numel() - 1
    out = torch.zeros(E, x.shape[1], g.shape[1], dtype=torch.float64)
    size = torch.zeros_like(out)
    for e in range(E):
        of = slice(int(offsets[e]), int(offsets[e + 1]))
        out[e] = x[of].T @ g[of].double()
        size[e] = x[of].T.abs() @ g[of].double().abs()
    return out, size


def weight_grad_bound(out, size, offsets, dtype):
    """Three planes of a float32 gradient, two of a float16 one; parts of 256 rows and more are added in turn."""
    planes = {torch.float32: 3, torch.float16: 2, torch.bfloat16: 1}[dtype]
    rows = (offsets[1:] - offsets[:-1]).double()[:, None, None]
    return (planes * (rows / 16 + 2) + 16 + rows / 256 + 2) * STEP * size + rounding(out, torch.float32)
