"""Layer norm and its backward against the 64-bit forms, within bounds that count float32 roundings."""
import pytest
import torch

import train_util as tu
from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def inputs(rows, dim, dtype, wdtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, dim, generator=g) * torch.exp(0.5 * torch.randn(dim, generator=g)) + 3.0
    w, b = 1 + 0.1 * torch.randn(dim, generator=g), 0.1 * torch.randn(dim, generator=g)
    gy = torch.randn(rows, dim, generator=g)
    return x.to(dtype), w.to(wdtype), b.to(wdtype), gy.to(dtype)


def off_by(t, elements):
    """A contiguous device copy of t that starts `elements` elements into its allocation."""
    flat = torch.zeros(t.numel() + elements, dtype=t.dtype, device="cuda")
    flat[elements:] = t.reshape(-1).cuda()
    return flat[elements:].view(t.shape)


def check_forward(x, w, b, out):
    y, mean, rstd = tu.layer_norm(x, w, b, EPS)
    by, bm, br = tu.layer_norm_bound(x, w, b, EPS, x.dtype)
    tu.assert_within(out.mean, mean, bm, "mean")
    tu.assert_within(out.rstd, rstd, br, "rstd")
    tu.assert_within(out.y, y, by, "y")


def check_backward(x, w, mean, rstd, gy, out):
    want = tu.layer_norm_grad(x, w, mean, rstd, gy)
    bound = tu.layer_norm_grad_bound(x, w, mean, rstd, gy)
    for name, got, e, t in zip(("x", "weight", "bias"), (out.x, out.weight, out.bias), want, bound):
        tu.assert_within(got, e, t, f"grad {name}")


# every way a row is held (lanes and packs of each type) and its edges, odd widths, one column, one row
SIZES = [(1, 1), (3, 2), (5, 63), (7, 64), (33, 128), (9, 129), (4, 512), (6, 513), (257, 500), (3, 1024), (5, 1025),
         (2, 2048), (3, 2049), (2, 4096), (3, 4097), (1, 8192), (2, 8195), (1, 20001), (2050, 77), (1030, 769)]


@pytest.mark.parametrize("types", ["f32", "bf16", "f16", "bf16/f32", "f16/f32"])
@pytest.mark.parametrize("rows,dim", SIZES)
def test_forward_and_backward(rows, dim, types):
    dtype, wdtype = tu.DTYPES[types.split("/")[0]], tu.DTYPES[types.split("/")[-1]]
    x, w, b, gy = inputs(rows, dim, dtype, wdtype, seed=rows * 31 + dim)
    dx, dw, db, dgy = (t.cuda() for t in (x, w, b, gy))
    out = binding.gs_layer_norm_fwd(dx, dw, db, eps=EPS)
    check_forward(x, w, b, out)
    grad = binding.gs_layer_norm_bwd(dx, dw, out.mean, out.rstd, dgy)
    check_backward(x, w, out.mean.cpu(), out.rstd.cpu(), gy, grad)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shift", [1, 3])
def test_any_alignment(name, shift):
    dtype = tu.DTYPES[name]
    x, w, b, gy = inputs(19, 1016, dtype, dtype, seed=shift)
    dx, dw, db, dgy = (off_by(t, shift) for t in (x, w, b, gy))
    out = binding.LayerNorm(off_by(x, shift + 1), torch.empty(19, device="cuda"), torch.empty(19, device="cuda"))
    binding.gs_layer_norm_fwd(dx, dw, db, eps=EPS, out=out)
    check_forward(x, w, b, out)
    grad = binding.LayerNormGrad(off_by(x, shift), off_by(w, 1), off_by(b, 1))
    binding.gs_layer_norm_bwd(dx, dw, out.mean, out.rstd, dgy, out=grad)
    check_backward(x, w, out.mean.cpu(), out.rstd.cpu(), gy, grad)


def test_outputs_end_where_they_should():
    """The elements before and after each output keep their values."""
    for dtype in tu.DTYPES.values():
        x, w, b, gy = inputs(5, 1003, dtype, dtype)
        room = [torch.full((n + 16,), 7.0, dtype=t, device="cuda")
                for n, t in ((5 * 1003, dtype), (5, torch.float32), (5, torch.float32), (5 * 1003, dtype),
                             (1003, dtype), (1003, dtype))]
        inner = [r[8:-8] for r in room]
        out = binding.LayerNorm(inner[0].view(5, 1003), inner[1], inner[2])
        binding.gs_layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), out=out)
        binding.gs_layer_norm_bwd(x.cuda(), w.cuda(), out.mean, out.rstd, gy.cuda(),
                                  out=binding.LayerNormGrad(inner[3].view(5, 1003), inner[4], inner[5]))
        for r in room:
            assert (r[:8] == 7).all() and (r[-8:] == 7).all()
        check_forward(x, w, b, out)


def test_no_bias_no_stats_no_rows_and_leading_axes():
    x, w, b, gy = inputs(6, 200, torch.float32, torch.float32)
    full = binding.gs_layer_norm_fwd(x.cuda(), w.cuda(), torch.zeros(200, device="cuda"))
    out = binding.gs_layer_norm_fwd(x.cuda().view(2, 3, 200), w.cuda(), stats=False)
    assert out.mean is None and out.rstd is None and out.y.shape == (2, 3, 200)
    assert torch.equal(out.y.view(6, 200), full.y)
    grad = binding.gs_layer_norm_bwd(x.cuda().view(2, 3, 200), w.cuda(), full.mean.view(2, 3), full.rstd.view(2, 3),
                                     gy.cuda().view(2, 3, 200), grad_bias=False)
    both = binding.gs_layer_norm_bwd(x.cuda(), w.cuda(), full.mean, full.rstd, gy.cuda())
    assert grad.bias is None and torch.equal(grad.weight, both.weight) and torch.equal(grad.x.view(6, 200), both.x)
    none = torch.zeros(0, 200, device="cuda")
    out = binding.gs_layer_norm_fwd(none, w.cuda(), b.cuda())
    assert out.y.shape == (0, 200) and out.mean.shape == (0,)
    grad = binding.gs_layer_norm_bwd(none, w.cuda(), out.mean, out.rstd, none)
    assert grad.x.shape == (0, 200) and not grad.weight.any() and not grad.bias.any()


def test_constant_rows_and_rows_that_are_not_finite():
    """A constant row gives the bias exactly; a row with an infinity or NaN spoils no other row."""
    x, w, b, gy = inputs(9, 777, torch.float32, torch.float32)
    x[2] = 5.0
    x[4, 100], x[6, 3] = float("inf"), float("nan")
    out = binding.gs_layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    y = out.y.cpu()
    assert torch.equal(y[2], b) and out.mean[2].item() == 5.0
    for r in (4, 6):
        assert y[r].isnan().all()
    keep = [r for r in range(9) if r not in (4, 6)]
    good = binding.LayerNorm(out.y[keep], out.mean[keep], out.rstd[keep])
    check_forward(x[keep], w, b, good)
    grad = binding.gs_layer_norm_bwd(x.cuda(), w.cuda(), out.mean, out.rstd, gy.cuda())
    got = grad.x.cpu()
    assert got[4].isnan().all() and got[6].isnan().all() and grad.weight.isnan().all()
    want = tu.layer_norm_grad(x[keep], w, good.mean.cpu(), good.rstd.cpu(), gy[keep])[0]
    bound = tu.layer_norm_grad_bound(x[keep], w, good.mean.cpu(), good.rstd.cpu(), gy[keep])[0]
    tu.assert_within(got[keep], want, bound, "grad x")


def test_rows_far_from_zero_keep_their_variance():
    """Values of 1000 with a spread of 0.01: a variance formed as mean(x^2) - mean^2 would lose it."""
    g = torch.Generator().manual_seed(4)
    x = 1000 + 0.01 * torch.randn(8, 4096, generator=g)
    w, b = torch.ones(4096), torch.zeros(4096)
    check_forward(x, w, b, binding.gs_layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), eps=EPS))


def test_gradient_against_differences_of_the_forward():
    """The gradient's products with directions against central differences of the 64-bit forward."""
    x, w, b, gy = inputs(6, 300, torch.float32, torch.float32, seed=9)
    out = binding.gs_layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    grad = binding.gs_layer_norm_bwd(x.cuda(), w.cuda(), out.mean, out.rstd, gy.cuda())
    g = torch.Generator().manual_seed(10)
    loss = lambda x, w, b: (gy.double() * tu.layer_norm(x, w, b, EPS)[0]).sum().item()  # noqa: E731
    bounds = tu.layer_norm_grad_bound(x, w, out.mean.cpu(), out.rstd.cpu(), gy)
    for i, (got, bound) in enumerate(zip((grad.x, grad.weight, grad.bias), bounds)):
        at = [x.double(), w.double(), b.double()]
        d = torch.randn(at[i].shape, generator=g, dtype=torch.float64)
        h = 1e-6
        at[i] = at[i] + h * d
        up = loss(*at)
        at[i] = at[i] - 2 * h * d
        down = loss(*at)
        # the statistics that the backward is given are off by float32 roundings too: 2^-20 of the terms' size
        got = got.cpu().double()
        room = (bound * d.abs()).sum().item() + 2.0 ** -20 * (got * d).abs().sum().item() + 1e-6
        assert abs((got * d).sum().item() - (up - down) / (2 * h)) <= room


def test_same_bits_on_a_side_stream_and_again():
    x, w, b, gy = (t.cuda() for t in inputs(4100, 640, torch.bfloat16, torch.float32))
    out = binding.gs_layer_norm_fwd(x, w, b)
    grad = binding.gs_layer_norm_bwd(x, w, out.mean, out.rstd, gy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        o = binding.gs_layer_norm_fwd(x, w, b, stream=side)
        q = binding.gs_layer_norm_bwd(x, w, o.mean, o.rstd, gy, stream=side)
        side.synchronize()
        for got, want in ((o.y, out.y), (o.mean, out.mean), (o.rstd, out.rstd), (q.x, grad.x),
                          (q.weight, grad.weight), (q.bias, grad.bias)):
            assert torch.equal(got, want)


def test_captured_into_a_graph():
    x, w, b, gy = (t.cuda() for t in inputs(300, 1000, torch.float32, torch.float32))
    out = binding.gs_layer_norm_fwd(x, w, b)
    grad = binding.gs_layer_norm_bwd(x, w, out.mean, out.rstd, gy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = binding.gs_layer_norm_fwd(x, w, b)
        q = binding.gs_layer_norm_bwd(x, w, o.mean, o.rstd, gy)
    for k in range(3):
        x.add_(0.5 * k)
        want = binding.gs_layer_norm_fwd(x, w, b)
        wgrad = binding.gs_layer_norm_bwd(x, w, want.mean, want.rstd, gy)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, e in ((o.y, want.y), (q.x, wgrad.x), (q.weight, wgrad.weight), (q.bias, wgrad.bias)):
            assert torch.equal(got, e)


def test_more_elements_than_32_bits_count():
    """A batch of 2^31 + 2^16 elements: the last rows are written and right."""
    rows, dim = (1 << 19) + 16, 4096
    x = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    w, b = torch.ones(dim, dtype=torch.bfloat16), torch.zeros(dim, dtype=torch.bfloat16)
    out = binding.gs_layer_norm_fwd(x, w.cuda(), b.cuda(), eps=EPS)
    last = slice(rows - 20, rows)
    check_forward(x[last].cpu(), w, b, binding.LayerNorm(out.y[last], out.mean[last], out.rstd[last]))
    grad = binding.gs_layer_norm_bwd(x, w.cuda(), out.mean, out.rstd, out.y)
    args = (x[last].cpu(), w, out.mean[last].cpu(), out.rstd[last].cpu(), out.y[last].cpu())
    tu.assert_within(grad.x[last], tu.layer_norm_grad(*args)[0], tu.layer_norm_grad_bound(*args)[0], "grad x")
