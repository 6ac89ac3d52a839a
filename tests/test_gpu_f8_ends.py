"""Products and weight gradients of 8-bit values at both ends of their scales: every number of e4m3 under scales from the
least to the largest, finite inputs next to float32's end, and float32 gradients down to its least number."""
import pytest
import torch

import train_util as tu
from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu
CODES = torch.tensor([c for c in range(256) if c % 128 != 127], dtype=torch.uint8)  # the numbers among them
NUMBERS = CODES.view(torch.float8_e4m3fn).double()
ONE = 0x38
BYTES = [1, 2, 3, 4, 20, 100, 127, 200, 240, 246, 247, 248, 251, 254]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def rows_of(codes, byte, place):
    """A row for each code, which stands at `place` of 300 columns; the other blocks have another scale."""
    values, scales = torch.zeros(len(codes), 384, dtype=torch.uint8), torch.full((len(codes), 3), 90, dtype=torch.uint8)
    values[:, place] = codes
    scales[:, place // 128] = byte
    return binding.Quantized(values.view(torch.float8_e4m3fn).cuda(), scales.cuda(), 300)


def as_bfloat16(v):
    """The nearest bfloat16, the largest beyond its range."""
    most = torch.finfo(torch.bfloat16).max
    return v.clamp(-most, most).float().bfloat16().double()


@pytest.mark.parametrize("byte", BYTES)
@pytest.mark.parametrize("place", [0, 200, 299])
def test_products(byte, place):
    """Next to a weight of the opposite scale: every result is of normal size, and exact."""
    other = min(254, max(1, 254 - byte))
    x, w = rows_of(CODES, byte, place), rows_of(torch.tensor([ONE, ONE + 128], dtype=torch.uint8), other, place)
    v, sign = NUMBERS * 2.0 ** (byte - 127), torch.tensor([1.0, -1.0], dtype=torch.float64)
    for name, dtype in tu.DTYPES.items():
        got = binding.gs_expert_product(x, w, dtype=dtype).cpu()
        taken = as_bfloat16(v) if name == "f32" else v
        want = taken[:, None] * 2.0 ** (other - 127) * sign
        assert torch.equal(got.double() + 0.0, want.to(dtype).double() + 0.0), name


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("byte", BYTES)
@pytest.mark.parametrize("cols", [254, 1003])
def test_weight_gradients(byte, cols, name):
    """One number times one number a column: exact, and zeros stay zeros."""
    power = max(-126, min(127, 127 - byte)) if name != "f16" else max(-14, min(15, 127 - byte))
    place = 200
    x, v = rows_of(CODES, byte, place), as_bfloat16(NUMBERS * 2.0 ** (byte - 127))
    grad = torch.zeros(len(CODES), cols)
    grad[:, :len(CODES)].fill_diagonal_(2.0 ** power)
    got = binding.gs_expert_weight_grad(x, grad.to(tu.DTYPES[name]).cuda()).cpu().double()
    want = torch.zeros(300, cols, dtype=torch.float64)
    want[place, :len(CODES)] = (v * 2.0 ** power).float().double()
    assert torch.equal(got + 0.0, want + 0.0)


@pytest.mark.parametrize("dim,cols", [(300, 40), (1100, 1032)])
def test_finite_inputs_stay_finite(dim, cols):
    """The largest numbers of float32 in one place a row, ordinary ones elsewhere: nothing that is not theirs changes, and
    theirs are the largest bfloat16 times what they meet, zeros among it."""
    g = torch.Generator().manual_seed(dim)
    rows, experts = 700, 30
    ids = torch.randint(0, experts, (rows, 1), generator=g, dtype=torch.int32)
    offsets, _, pairs = tu.expert_plan(ids, experts)
    plan = binding.gs_expert_plan(ids.cuda(), experts)
    x = torch.zeros(rows, dim)
    x[:, 128:] = torch.randint(-3, 4, (rows, dim - 128), generator=g).float()
    x[::3, 5] = torch.finfo(torch.float32).max
    x[1::3, 7] = -3.4e38
    grad = torch.randint(-1, 2, (rows, cols), generator=g).float() * 2.0 ** -20
    q = binding.gs_quantize(x.cuda())
    most = torch.finfo(torch.bfloat16).max
    taken = x.double().clamp(-most, most)
    for name, dtype in tu.DTYPES.items():
        got = binding.gs_expert_weight_grad(q, grad.to(dtype).cuda(), plan, gather=True).cpu().double()
        for e in range(experts):
            at = slice(int(offsets[e]), int(offsets[e + 1]))
            mine, met = taken[pairs[at].long()].T, grad[at].double()  # the gradient's rows are the sorted ones
            want = mine @ met
            # sums of at most 40 terms of one size, or exact
            near = (got[e] - want).abs() <= 40 * tu.U * (mine.abs() @ met.abs())
            assert near.all(), (name, e)
            assert torch.equal(got[e][128:], want[128:])
    w = torch.zeros(50, dim)
    w[:, 128:] = torch.randint(-3, 4, (50, dim - 128), generator=g).float()
    w[0, 5], w[1, 7] = 2.0 ** -20, 2.0 ** -20
    got = binding.gs_expert_product(q, binding.gs_quantize(w.cuda()), dtype=torch.float32).cpu().double()
    want = taken @ w.double().T
    assert torch.equal(got[:, 2:], want[:, 2:])
    near = (got - want).abs() <= 8 * tu.U * (taken.abs() @ w.double().T.abs())
    assert near.all()


def test_no_number_beside_the_largest():
    """A NaN stays one where the largest numbers are taken in place of infinities."""
    x = torch.zeros(40, 128)
    x[0, 0], x[1, 1], x[2, 2] = torch.finfo(torch.float32).max, float("nan"), float("inf")
    q = binding.gs_quantize(x.cuda())
    q.scales[:, 0] = 247
    got = binding.gs_expert_product(q, binding.gs_quantize(torch.eye(3, 128).cuda()), dtype=torch.float32).cpu()
    assert torch.equal(got.isnan(), torch.tensor([[t in (1, 2)] * 3 for t in range(40)])) and got[0, 0].isfinite()
    grad = torch.ones(40, 4)
    got = binding.gs_expert_weight_grad(q, grad.cuda()).cpu()
    assert torch.equal(got.isnan().any(dim=1), torch.tensor([k in (1, 2) for k in range(128)]))


@pytest.mark.parametrize("exponent", [-149, -140, -134, -133, -127, -126, -118, -111, -110, -109, -80, 0, 100])
def test_small_float32_gradients(exponent):
    """24 bits from 2^-110 on; below, less than 2^-133 is cut off, towards zero."""
    g = torch.Generator().manual_seed(1)
    q = binding.gs_quantize(torch.full((1, 1), 1.0, device="cuda"))
    grad = (1 + torch.rand(1, 500, generator=g)) * 2.0 ** exponent
    grad = torch.cat([grad, -grad], dim=1)
    got = binding.gs_expert_weight_grad(q, grad.cuda()).cpu().double()
    less = grad.double().abs() - got.abs()
    assert (less >= 0).all() and (less < 2.0 ** -133).all() and (got * grad.double() >= 0).all()
    if exponent >= -110:
        assert (less == 0).all()
