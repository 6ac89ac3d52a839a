"""Plain 64-bit forms of the training operators (CPU tensors) and the error bounds their GPU results are held to.

The bounds count roundings: one rounding to type t is off by at most half a step, eps(t) / 2 relative to the value (and
by half the smallest subnormal where the value is below the type's normal range); a float32 sum of n terms, added in
chains of at most d additions, is off by at most d * 2^-24 * sum |terms|, and one more 2^-24 of a term for each
operation that forms it.
"""
import torch

U = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def rounding(value, dtype):
    """Half a step of dtype around each value, with 2 * 2^-24 for the value's own last float32 operations."""
    return (torch.finfo(dtype).eps / 2 + 2 * U) * value.abs() + TINY[dtype]


def assert_within(got, want, bound, what):
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    finite = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), finite), f"{what}: other entries are finite"
    off = torch.where(finite, (got - want).abs() - bound, torch.full_like(want, -1.0))
    assert not off.numel() or not (off > 0).any(), \
        f"{what}: {int((off > 0).sum())} of {off.numel()} beyond the bound, worst by {off.max().item():.3g}"


# ----------------------------------------------------------------------------------------------------------------
# layer norm


def layer_norm(x, weight, bias, eps):
    """(y, mean, rstd) of float64 rows [R, D]."""
    x, w = x.double(), weight.double()
    mean = x.mean(dim=1)
    c = x - mean[:, None]
    rstd = (c.square().mean(dim=1) + eps).rsqrt()
    y = c * rstd[:, None] * w
    return (y if bias is None else y + bias.double()), mean, rstd


def layer_norm_bound(x, weight, bias, eps, out_dtype):
    """Bounds of y, mean and rstd. A row's sums are chains of at most 32 additions in a lane (or D / 256 where the row
    is read in pieces) and 12 across lanes."""
    y, mean, rstd = layer_norm(x, weight, bias, eps)
    x, w = x.double(), weight.double()
    depth = 48 + x.shape[1] / 256
    e_mean = (depth + 2) * U * x.abs().mean(dim=1)
    c = (x - mean[:, None]).abs()
    e_c = e_mean[:, None] + U * (c + e_mean[:, None])
    # of the mean square: its own sum, and the error of c in first and second order
    e_q = (depth + 2) * U * c.square().mean(dim=1) + (2 * c * e_c + e_c.square()).mean(dim=1)
    rel = e_q * rstd.square() / 2 * (1 + 2 * e_q * rstd.square()) + 4 * U
    e_y = w.abs() * rstd[:, None] * (e_c * (1 + rel[:, None]) + c * (rel[:, None] + 3 * U))
    return e_y * (1 + 4 * U) + rounding(y, out_dtype), e_mean + 1e-300, rel * rstd


def layer_norm_grad(x, weight, mean, rstd, grad_y):
    x, w, g = x.double(), weight.double(), grad_y.double()
    xh = (x - mean.double()[:, None]) * rstd.double()[:, None]
    gw = g * w
    gx = rstd.double()[:, None] * (gw - gw.mean(dim=1, keepdim=True) - xh * (gw * xh).mean(dim=1, keepdim=True))
    return gx, (g * xh).sum(dim=0), g.sum(dim=0)


def layer_norm_grad_bound(x, weight, mean, rstd, grad_y):
    """Column sums are chains of at most rows / 64 additions in a workgroup, and 64 more to join them."""
    gx, gw, gb = layer_norm_grad(x, weight, mean, rstd, grad_y)
    R, D = x.shape
    rs = rstd.double()[:, None]
    xh = ((x.double() - mean.double()[:, None]) * rs).abs()
    g = grad_y.double().abs()
    gwt = g * weight.double().abs()
    depth, depth_r = 48 + D / 256, 96 + R / 64
    e_s1 = (depth + 3) * U * gwt.mean(dim=1, keepdim=True)
    e_s2 = (depth + 6) * U * (gwt * xh).mean(dim=1, keepdim=True)
    s1 = (grad_y.double() * weight.double()).mean(dim=1, keepdim=True).abs()
    s2 = (gwt * xh).mean(dim=1, keepdim=True)
    e_gx = rs * (4 * U * gwt + e_s1 + 3 * U * s1 + xh * (e_s2 + 6 * U * s2))
    e_gw = (depth_r + 4) * U * (g * xh).sum(dim=0)
    e_gb = (depth_r + 1) * U * g.sum(dim=0)
    return (e_gx + rounding(gx, x.dtype), e_gw + rounding(gw, weight.dtype), e_gb + rounding(gb, weight.dtype))


# ----------------------------------------------------------------------------------------------------------------
# experts


def expert_plan(ids, experts):
    """(offsets, rows, pairs) of int32 ids [T, K] by counting, pair by pair."""
    flat = ids.reshape(-1).tolist()
    lists = [[] for _ in range(experts)]
    for p, e in enumerate(flat):
        if 0 <= e < experts:
            lists[e].append(p)
    rows, pairs, offsets = [-1] * len(flat), [], [0]
    for of in lists:
        for p in of:
            rows[p] = len(pairs)
            pairs.append(p)
        offsets.append(len(pairs))
    pairs += [-1] * (len(flat) - len(pairs))
    return (torch.tensor(offsets, dtype=torch.int32), torch.tensor(rows, dtype=torch.int32).reshape(ids.shape),
            torch.tensor(pairs, dtype=torch.int32))


def expert_dispatch(x, pairs, choices):
    out = torch.zeros(pairs.numel(), x.shape[1], dtype=x.dtype)
    kept = pairs >= 0
    out[kept] = x[(pairs[kept] // choices).long()]
    return out


def expert_combine(source, rows, weights):
    """(y, sum of magnitudes)."""
    T, K = rows.shape
    y = torch.zeros(T, source.shape[1], dtype=torch.float64)
    size = torch.zeros_like(y)
    for k in range(K):
        kept = rows[:, k] >= 0
        term = source[rows[kept, k].long()].double()
        if weights is not None:
            term = term * weights[kept, k].double()[:, None]
        y[kept] += term
        size[kept] += term.abs()
    return y, size


def expert_combine_bound(source, rows, weights):
    y, size = expert_combine(source, rows, weights)
    return (rows.shape[1] + 1) * U * size + rounding(y, source.dtype)


def expert_combine_grad(source, rows, weights, grad_y):
    """(grad_source, grad_weights, sum of magnitudes of grad_weights)."""
    T, K = rows.shape
    gs = torch.zeros(source.shape, dtype=torch.float64)
    gw = torch.zeros(T, K, dtype=torch.float64)
    size = torch.zeros_like(gw)
    for k in range(K):
        kept = rows[:, k] >= 0
        at = rows[kept, k].long()
        g = grad_y[kept].double()
        gs[at] = g * weights[kept, k].double()[:, None]
        gw[kept, k] = (g * source[at].double()).sum(dim=1)
        size[kept, k] = (g * source[at].double()).abs().sum(dim=1)
    return gs, gw, size


# ----------------------------------------------------------------------------------------------------------------
# orthogonalised update

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def operand_bits(dtype, rows, left):
    """Bits that a step's three products keep of their operands (the Gram product, its square, the product with X):
    both halves, 22, or the high halves, 11. rows: of the smaller side; left: steps left, this one among them."""
    if dtype == torch.float32 or rows <= 736:  # padded to 32, below 768
        return 22, 22, 22
    if left > (3 if dtype == torch.float16 else 2):
        return 11, 11, 11
    return (22, 22, 22) if dtype == torch.float16 else (11, 22, 22)


def orthogonalize(update, steps=5, coefficients=COEFFICIENTS, eps=1e-7, noise=None):
    """The result for one matrix in 64 bits; with noise (a generator) the same with every rounding that the kernels
    make replaced by a random one of its size."""
    a, b, c = coefficients
    x = update.double()
    x = x / (x.norm() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T.contiguous() if tall else x
    K = max(x.shape)

    def near(v, relative):
        return v if noise is None else v * (1 + relative * (2 * torch.rand(v.shape, generator=noise,
                                                                            dtype=torch.float64) - 1))

    def product(p, q, bits):
        # a rounding of each operand to `bits` bits, and a float32 sum of K terms, 16 at a time and 3 products each:
        # its roundings are of partial sums, at most the size of |p| |q|
        out = near(p, 2.0 ** -bits) @ near(q, 2.0 ** -bits)
        if noise is not None:
            size = (K * 3 / 16 + 16) ** 0.5 * U * (p.norm(dim=1)[:, None] * q.norm(dim=0)[None, :])
            out = out + size * (2 * torch.rand(out.shape, generator=noise, dtype=torch.float64) - 1)
        return out

    x = near(x, 2.0 ** -22)
    for s in range(steps):
        gram, square, apply = operand_bits(update.dtype, min(x.shape), steps - s)
        A = near(product(x, x.T.contiguous(), gram), 2.0 ** -22)
        B = near(b * A + c * product(A, A, square), 2.0 ** -22)
        x = near(a * x + product(B, x, apply), 2.0 ** -22)
    return x.T.contiguous() if tall else x


def orthogonalize_bound(update, want, seed=0, **kw):
    """(entry by entry, 2-norm): four times what three runs with random roundings are off by at most, plus the
    rounding of the result. An entry's bound is four of the largest entry's in those runs: their own size varies
    little from entry to entry."""
    worst, norm = 0.0, 0.0
    for k in range(3):
        g = torch.Generator().manual_seed(seed + k)
        d = orthogonalize(update, noise=g, **kw) - want
        worst, norm = max(worst, d.abs().max().item()), max(norm, d.norm().item())
    r = rounding(want, update.dtype)
    return 4 * worst + r, 4 * norm + r.norm().item()
