"""Products whose blocks all have scales of their own, one block of a row at a time: whole numbers, so every result is exact,
and another block's scale would show. In each kernel's tiles, by the rule that the entry point states beside its launches."""
import pytest
import torch

import train_util as tu
from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu
UNITS = 256


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def tile(rows, experts, blocks, cols):
    """Edge of the tiles that 16-bit results take."""
    if blocks >= 16 and rows // experts >= 512 and rows // 256 * -(-cols // 256) >= UNITS:
        return 256
    return 64 if rows // 128 * -(-cols // 128) < UNITS else 128


def check(counts, past, dim, cols, names, seed, far):
    """far: the blocks' scales lie up to 2^far apart, x's and the weight's in opposite directions."""
    g = torch.Generator().manual_seed(seed)
    off = torch.tensor([0] + counts).cumsum(0).int()
    T, E, blocks = int(off[-1]) + past, len(counts), -(-dim // 128)
    token = torch.randperm(T, generator=g)
    plan = binding.ExpertPlan(off.cuda(), torch.zeros(T, 1, dtype=torch.int32, device="cuda"), token.int().cuda())
    base = torch.randint(-far, far + 1, (blocks,), generator=g)
    scale_x = base + torch.randint(-3, 4, (T, blocks), generator=g)
    scale_w = -base + torch.randint(-3, 4, (E, cols, blocks), generator=g)
    # x: one block a row, its others zeros under scales that would show
    block = torch.randint(0, blocks, (T,), generator=g)
    x = torch.randint(-3, 4, (T, 128), generator=g).float()
    last = dim - (blocks - 1) * 128
    x[block == blocks - 1, last:] = 0
    full = torch.zeros(T, blocks, 128)
    full[torch.arange(T), block] = x
    w = torch.randint(-3, 4, (E, cols, blocks, 128), generator=g).float()
    w[:, :, -1, last:] = 0
    held = [binding.Quantized(v.flatten(-2).to(torch.float8_e4m3fn).cuda(), (s + 127).to(torch.uint8).cuda(), dim)
            for v, s in ((full, scale_x), (w, scale_w))]
    got = {name: binding.gs_expert_product(*held, plan, gather=True, dtype=tu.DTYPES[name]).cpu() for name in names}
    picked = [r for e in range(E) for r in range(int(off[e]), int(off[e + 1]))
              if T < 2000 or (r - int(off[e])) % 64 in (0, 1, 31, 37, 63) or r == int(off[e + 1]) - 1]
    expert = torch.searchsorted(off[1:].long(), torch.tensor(picked), right=True)
    for e in range(E):
        rows = torch.tensor(picked)[expert == e]
        for b in range(blocks):
            mine = rows[block[token[rows]] == b]
            if len(mine) == 0:
                continue
            t = token[mine]
            want = (x[t].double() @ w[e, :, b].double().T) * torch.exp2(
                (scale_x[t, b][:, None] + scale_w[e, :, b][None]).double())
            for name in names:
                assert torch.equal(got[name][mine].double(), want.to(tu.DTYPES[name]).double()), (name, e, b)
    for name in names:
        assert (got[name][int(off[-1]):] == 0).all()


# blocks below and above the 32 whose scales are held at once, whole words of four of them and not
@pytest.mark.parametrize("dim", [100, 128 * 3, 128 * 7 + 1, 128 * 32, 128 * 33 + 5, 128 * 70])
def test_smallest_tiles(dim):
    counts, cols = [33, 0, 1, 70, 64], 75
    assert tile(sum(counts) + 9, 5, -(-dim // 128), cols) == 64
    check(counts, 9, dim, cols, ["f32", "bf16", "f16"], dim, 4)
    check(counts, 9, dim, cols, ["f32", "bf16"], dim, 90)


@pytest.mark.parametrize("dim", [300, 128 * 15, 128 * 37])
def test_middle_tiles(dim):
    counts, cols = [1500, 0, 1, 1300, 1129], 1029
    assert tile(sum(counts) + 9, 5, -(-dim // 128), cols) == 128
    check(counts, 9, dim, cols, ["f32", "bf16", "f16"], dim, 4)
    check(counts, 9, dim, cols, ["bf16"], dim, 90)


@pytest.mark.parametrize("dim", [128 * 16, 128 * 18 + 77, 128 * 34 + 1])
def test_largest_tiles(dim):
    counts, cols = [6001, 1, 0, 4600, 6107], 1029
    assert tile(sum(counts) + 77, 5, -(-dim // 128), cols) == 256
    check(counts, 77, dim, cols, ["bf16", "f16"], dim, 4)
    check(counts, 77, dim, cols, ["bf16"], dim, 90)
