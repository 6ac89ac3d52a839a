"""Values held in 8 bits, bit by bit against rounding in 64 bits, and the products of such values within bounds that count
float32 roundings."""
import pytest
import torch

import f8_util as fu
import train_util as tu
from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def same_numbers(got, want):
    got, want = got.cpu().double(), want.double()
    assert got.shape == want.shape
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


def check_held(x, transpose=False, place=lambda t: t.cuda()):
    got = binding.gs_quantize(place(x), transpose=transpose)
    values, scales = fu.quantize(x.transpose(-1, -2) if transpose else x)
    assert torch.equal(got.scales.cpu(), scales)
    same_numbers(got.values.float(), values)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        back = binding.gs_dequantize(got, dtype=dtype)
        most = torch.finfo(dtype).max
        want = fu.values_of(values, scales, got.dim)
        want = want.clamp(-most, most)
        assert back.dtype == dtype and back.shape == want.shape
        if dtype == torch.float16:  # what is below its range is rounded
            want = want.to(dtype).double()
        same_numbers(back.double(), want)
    return got


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1,), (127,), (3, 1), (5, 128), (2, 129), (7, 1001), (4, 3, 257), (300, 64), (1, 5000),
                                   (0, 40), (2, 0, 7)])
def test_held_values(shape, name):
    g = torch.Generator().manual_seed(sum(shape))
    x = torch.randn(shape, generator=g) * torch.exp(4 * torch.randn(shape[-1], generator=g))
    check_held(x.clamp(-6e4, 6e4).to(tu.DTYPES[name]))


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 1), (128, 32), (3, 40), (129, 31), (4, 257, 70), (2, 100, 1), (1000, 3)])
def test_held_columns(shape, name):
    g = torch.Generator().manual_seed(sum(shape))
    x = torch.randn(shape, generator=g) * torch.exp(2 * torch.randn(shape[-1], generator=g))
    check_held(x.to(tu.DTYPES[name]), transpose=True)


def test_every_16_bit_value():
    """Each bfloat16 and float16, in blocks of like size and in blocks that hold all sizes."""
    for dtype in (torch.bfloat16, torch.float16):
        x = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(dtype)
        check_held(x.view(512, 128))
        check_held(x.view(128, 512).T.contiguous())


def test_ends_of_float32():
    """Subnormals, the largest numbers, halves of a step both ways, infinities and NaN beside numbers, and zeros."""
    tiny, most = 2.0 ** -149, torch.finfo(torch.float32).max
    rows = [[tiny], [tiny * 3, 2.0 ** -126], [most, 1.0], [2.0 ** 127, most / 2], [0.0, -0.0], [448.0, 449.0],
            [448.0, 448.0000305], [1.75, -1.0625], [float("inf"), 3.0], [float("-inf"), float("nan")],
            [float("nan"), 2.0 ** -100], [2.0 ** -118 * 1.75], [2.0 ** -118 * 1.7500001],
            [256.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9 * 1.5]]
    x = torch.zeros(len(rows), 130)
    for i, r in enumerate(rows):
        x[i, :len(r)] = torch.tensor(r)
    check_held(x)
    check_held(x.T.contiguous(), transpose=True)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_rows_at_any_alignment(name):
    def place(t):
        flat = torch.zeros(t.numel() + 3, dtype=t.dtype, device="cuda")
        flat[3:] = t.reshape(-1).cuda()
        return flat[3:].view(t.shape)
    x = torch.randn(37, 333, generator=torch.Generator().manual_seed(5)).to(tu.DTYPES[name])
    check_held(x, place=place)
    check_held(x, transpose=True, place=place)


def setup(T, K, E, D, N, seed, dropped, gather):
    """(plan on the GPU, its offsets and pairs, x and weight as Quantized, the sorted rows' and the weights' numbers)."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    ids[torch.rand(T, K, generator=g) < dropped] = -1
    offsets, _, pairs = tu.expert_plan(ids, E)
    plan = binding.gs_expert_plan(ids.cuda(), E)
    x = torch.randn(T if gather else T * K, D, generator=g) * torch.exp(torch.randn(D, generator=g))
    w = torch.randn(E, N, D, generator=g) * torch.exp(torch.randn(E, N, 1, generator=g))
    qx, qw = binding.gs_quantize(x.cuda()), binding.gs_quantize(w.cuda())
    rows = fu.held(qx)
    return plan, offsets, pairs, qx, qw, fu.sorted_rows(rows, pairs, K) if gather else rows, fu.held(qw)


SIZES = [(1, 1, 1, 1, 1, 0.0), (1, 2, 8, 200, 130, 0.0), (5, 3, 4, 128, 128, 0.3), (16, 2, 8, 512, 256, 0.0),
         (70, 2, 3, 129, 33, 0.1), (200, 3, 60, 300, 257, 0.1), (129, 1, 1, 640, 127, 0.0), (500, 2, 2, 257, 300, 0.5),
         (300, 1, 5, 64, 500, 1.0), (33, 2, 200, 385, 65, 0.1), (1000, 2, 3, 100, 70, 0.05)]


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,K,E,D,N,dropped", SIZES)
def test_product(T, K, E, D, N, dropped, name):
    dtype = tu.DTYPES[name]
    for gather in (False, True):
        plan, offsets, _, qx, qw, rows, w = setup(T, K, E, D, N, T + D, dropped, gather)
        want, size, most = fu.product(rows, w, offsets)
        bound = fu.product_bound(want, size, most, D, dtype)
        out = torch.full((T * K, N), 7.0, dtype=dtype, device="cuda")
        got = binding.gs_expert_product(qx, qw, plan, gather=gather, dtype=dtype, out=out)
        tu.assert_within(got, want, bound, "out")
        assert (got[int(offsets[-1]):] == 0).all()
        again = binding.gs_expert_product(qx, qw, plan, gather=gather, dtype=dtype)
        assert torch.equal(again, got)
        got = binding.gs_expert_product(qx, qw, plan, gather=gather, dtype=dtype, relu=True)
        tu.assert_within(got, want.clamp(min=0), bound, "relu")
        assert (got >= 0).all()


# one and several tiles of every size, the blocks whose scales are held at once, and one more
@pytest.mark.parametrize("R,N,D", [(1, 1, 1), (1, 300, 5000), (31, 64, 4096), (128, 128, 128), (257, 129, 4097),
                                   (700, 520, 256), (2000, 300, 130)])
def test_product_of_one_weight(R, N, D):
    g = torch.Generator().manual_seed(R)
    qx = binding.gs_quantize(torch.randn(R, D, generator=g).cuda())
    qw = binding.gs_quantize((torch.randn(N, D, generator=g) * torch.exp(torch.randn(D, generator=g))).cuda())
    want, size, most = fu.product(fu.held(qx), fu.held(qw)[None], torch.tensor([0, R]))
    for dtype in (torch.float32, torch.bfloat16):
        got = binding.gs_expert_product(qx, qw, dtype=dtype)
        tu.assert_within(got, want, fu.product_bound(want, size, most, D, dtype), "out")


def whole_numbers(g, *shape):
    return torch.randint(-7, 8, shape, generator=g).float()


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,K,E,D,N,dropped", SIZES + [(4000, 2, 4, 200, 300, 0.1), (2, 2, 8, 4225, 520, 0.0)])
def test_products_without_rounding(T, K, E, D, N, dropped, name):
    """Whole numbers up to 7: their products and sums are exact in every step, so that each term shows."""
    g = torch.Generator().manual_seed(T + N)
    ids = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    ids[torch.rand(T, K, generator=g) < dropped] = -1
    offsets, _, pairs = tu.expert_plan(ids, E)
    plan = binding.gs_expert_plan(ids.cuda(), E)
    x, w, grad = whole_numbers(g, T, D), whole_numbers(g, E, N, D), whole_numbers(g, T * K, N)
    qx, qw = binding.gs_quantize(x.cuda()), binding.gs_quantize(w.cuda())
    dtype = tu.DTYPES[name]
    rows = fu.sorted_rows(x, pairs, K).double()
    want = torch.zeros(T * K, N, dtype=torch.float64)
    for e in range(E):
        of = slice(int(offsets[e]), int(offsets[e + 1]))
        want[of] = rows[of] @ w[e].double().T
    got = binding.gs_expert_product(qx, qw, plan, gather=True, dtype=dtype)
    assert torch.equal(got.cpu(), want.to(dtype))
    got = binding.gs_expert_weight_grad(qx, grad.to(dtype).cuda(), plan, gather=True)
    assert torch.equal(got.cpu().double(), fu.weight_grad(rows, grad, offsets)[0])


def test_product_of_large_tiles():
    """As many rows and columns as the largest tiles take, uneven experts among them."""
    g = torch.Generator().manual_seed(1)
    T, K, E, D, N = 9000, 2, 3, 300, 1100
    ids = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    ids[: T // 3] = 1
    ids[torch.rand(T, K, generator=g) < 0.03] = -1
    offsets, _, pairs = tu.expert_plan(ids, E)
    plan = binding.gs_expert_plan(ids.cuda(), E)
    qx = binding.gs_quantize(torch.randn(T, D, generator=g).cuda())
    qw = binding.gs_quantize(torch.randn(E, N, D, generator=g).cuda())
    want, size, most = fu.product(fu.sorted_rows(fu.held(qx), pairs, K), fu.held(qw), offsets)
    got = binding.gs_expert_product(qx, qw, plan, gather=True)
    tu.assert_within(got, want, fu.product_bound(want, size, most, D, torch.bfloat16), "out")


def test_scales_over_the_whole_range():
    """Blocks from 2^-100 to 2^100 next to each other: a block's scale counts for itself alone, as its products do."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(40, 640, generator=g) * torch.exp2(torch.randint(-50, 51, (40, 5), generator=g).float()
                                                       ).repeat_interleave(128, dim=1)
    w = torch.randn(50, 640, generator=g) * torch.exp2(torch.randint(-50, 51, (50, 5), generator=g).float()
                                                       ).repeat_interleave(128, dim=1)
    qx, qw = binding.gs_quantize(x.cuda()), binding.gs_quantize(w.cuda())
    want, size, most = fu.product(fu.held(qx), fu.held(qw)[None], torch.tensor([0, 40]))
    got = binding.gs_expert_product(qx, qw, dtype=torch.float32)
    tu.assert_within(got, want, fu.product_bound(want, size, most, 640, torch.float32), "out")


def test_no_number_stays_in_its_row():
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn(70, 200, generator=g), torch.randn(90, 200, generator=g)
    x[5, 130], x[6, 0], w[80, 199] = float("nan"), float("inf"), float("nan")
    qx, qw = binding.gs_quantize(x.cuda()), binding.gs_quantize(w.cuda())
    for relu in (False, True):
        got = binding.gs_expert_product(qx, qw, relu=relu).cpu()
        bad = torch.zeros(70, 90, dtype=torch.bool)
        bad[5:7], bad[:, 80] = True, True
        assert torch.equal(got.isnan(), bad)
    grad = torch.randn(70, 30, generator=g)
    grad[50, 7] = float("inf")
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        got = binding.gs_expert_weight_grad(qx, grad.to(dtype).cuda()).cpu()
        bad = torch.zeros(200, 30, dtype=torch.bool)
        bad[130], bad[0], bad[:, 7] = True, True, True
        assert torch.equal(got.isfinite(), ~bad)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,K,E,D,N,dropped", SIZES)
def test_weight_grad(T, K, E, D, N, dropped, name):
    dtype = tu.DTYPES[name]
    for gather in (False, True):
        plan, offsets, _, qx, _, rows, _ = setup(T, K, E, D, 1, T + N, dropped, gather)
        g = torch.Generator().manual_seed(N)
        grad = torch.randn(T * K, N, generator=g).to(dtype)
        grad[int(offsets[-1]):] = float("nan")  # not read
        want, size = fu.weight_grad(rows, grad, offsets)
        got = binding.gs_expert_weight_grad(qx, grad.cuda(), plan, gather=gather,
                                               out=torch.full((E, D, N), 7.0, device="cuda"))
        tu.assert_within(got, want, fu.weight_grad_bound(want, size, offsets, dtype), "grad weight")
        assert torch.equal(binding.gs_expert_weight_grad(qx, grad.cuda(), plan, gather=gather), got)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R,D,N", [(0, 5, 6), (1, 1, 1), (5000, 128, 256), (20000, 130, 9), (3001, 300, 8)])
def test_weight_grad_of_many_rows(R, D, N, name):
    """Sums in parts, and none at all."""
    g = torch.Generator().manual_seed(R)
    qx = binding.gs_quantize(torch.randn(R, D, generator=g).cuda())
    grad = torch.randn(R, N, generator=g).to(tu.DTYPES[name])
    offsets = torch.tensor([0, R])
    want, size = fu.weight_grad(fu.held(qx), grad, offsets)
    got = binding.gs_expert_weight_grad(qx, grad.cuda())
    tu.assert_within(got, want[0], fu.weight_grad_bound(want, size, offsets, tu.DTYPES[name])[0], "grad weight")


def test_weight_grad_of_the_largest_numbers():
    """float32 gradients next to the type's largest value keep their 24 bits, and stay finite."""
    x = torch.zeros(64, 128)
    x[3, 5], x[40, 7] = 0.5, 0.25
    grad = torch.zeros(64, 4)
    grad[3], grad[40] = torch.finfo(torch.float32).max, -3.4e38
    got = binding.gs_expert_weight_grad(binding.gs_quantize(x.cuda()), grad.cuda()).cpu()
    assert (got[5] == torch.finfo(torch.float32).max * 0.5).all() and (got[7] == grad[40] * 0.25).all()
