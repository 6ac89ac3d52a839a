"""Weight gradients of experts with more rows than are looked up at once (1024), in every tile and split, and of blocks whose
scales all differ. Whole numbers, so every sum is exact and each row shows."""
import pytest
import torch

import train_util as tu
from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu
SEGMENT, UNITS = 1024, 256


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def tiles(dim, cols, edge):
    return -(-dim // edge) * -(-cols // edge)


def chosen(rows, experts, dim, cols):
    """(edge of a tile, rows of a part or None) that the entry point's rule gives, checked by its workspace."""
    need = binding.load_library().gs_expert_weight_grad_workspace_bytes(rows, experts, dim, cols)
    large = experts * tiles(dim, cols, 256)
    if cols >= 8 and (large >= 2 * UNITS or (large >= UNITS and rows >= 768 * experts)):
        assert need == 0
        return 256, None
    if need == 0:
        return 128, None
    items = need // (dim * cols * 4)
    want = 2 * UNITS // tiles(dim, cols, 128) - experts
    want = want if want >= experts else 4 * UNITS // tiles(dim, cols, 128) - experts
    chunk = max(256, -(-(-(-rows // want)) // 32) * 32)
    assert items == rows // chunk + experts
    return 128, chunk


def case(counts, past, choices, dim, cols, seed, gather):
    """(plan, its rows' tokens, x as Quantized with scales of 2^-4 to 2^4, its numbers by sorted row, whole gradients)."""
    g = torch.Generator().manual_seed(seed)
    off = torch.tensor([0] + counts).cumsum(0).int()
    rows = int(off[-1]) + past
    assert rows % choices == 0
    pairs = torch.randperm(rows, generator=g).int()
    plan = binding.ExpertPlan(off.cuda(), torch.zeros(rows // choices, choices, dtype=torch.int32, device="cuda"),
                              torch.where(torch.arange(rows) < off[-1], pairs, -1).int().cuda())
    n = rows // choices if gather else rows
    blocks = -(-dim // 128)
    scale = torch.randint(-4, 5, (n, blocks), generator=g)
    whole = torch.randint(-3, 4, (n, blocks * 128), generator=g).float()
    whole[:, dim:] = 0
    q = binding.Quantized(whole.to(torch.float8_e4m3fn).cuda(), (scale + 127).to(torch.uint8).cuda(), dim)
    x = (whole.unflatten(1, (blocks, 128)) * torch.exp2(scale.float())[..., None]).flatten(1)[:, :dim]
    grad = torch.randint(-3, 4, (rows, cols), generator=g).float()
    return plan, off, q, x[(pairs // choices).long()] if gather else x, grad


def check(counts, past, choices, dim, cols, names, seed, gather=True):
    plan, off, q, x, grad = case(counts, past, choices, dim, cols, seed, gather)
    want = torch.stack([x[int(a):int(b)].T @ grad[int(a):int(b)] for a, b in zip(off[:-1], off[1:])])
    # multiples of 2^-4 up to 9 * 2^4 a row: whole in float32 up to 2^24 / 2304 rows, as long as no sum gets there
    assert want.abs().max() < 2.0 ** 20
    for name in names:
        grad_in = grad.to(tu.DTYPES[name])
        grad_in[int(off[-1]):] = float("nan")  # not read
        got = binding.gs_expert_weight_grad(q, grad_in.cuda(), plan, gather=gather).cpu()
        for e in range(len(counts)):
            assert torch.equal(got[e], want[e]), (name, e)


ROWS = [0, 1, SEGMENT - 1, SEGMENT, SEGMENT + 1, 3000, 2 * SEGMENT + 33, 700]


@pytest.mark.parametrize("cols", [1096, 1101, 1100])
@pytest.mark.parametrize("gather", [True, False])
def test_large_tiles_of_long_experts(cols, gather):
    """The tiles of 256 that long experts take, with widths of whole packs and widths that end inside one."""
    dim, past = 1700, 26
    rows = sum(ROWS) + past
    large = len(ROWS) * tiles(dim, cols, 256)
    assert UNITS <= large < 2 * UNITS and rows >= 768 * len(ROWS) and chosen(rows, len(ROWS), dim, cols) == (256, None)
    check(ROWS, past, 2, dim, cols, ["f32", "bf16", "f16"], cols, gather)


def test_large_tiles_of_many_matrices():
    """The same tiles because the matrices are many, one expert long."""
    counts, dim, cols = [2500 if e == 7 else 40 + e for e in range(36)], 900, 1030
    assert chosen(sum(counts), 36, dim, cols) == (256, None) and 36 * tiles(dim, cols, 256) >= 2 * UNITS
    check(counts, 0, 1, dim, cols, ["f32", "bf16", "f16"], 5)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("counts,cols", [([300001], 256), ([90001, 0, 1, 150000, 2047, 64000, 900, 1], 256),
                                         ([300001], 130), ([300000, 299999], 3)])
def test_parts_longer_than_a_segment(counts, cols, name):
    dim = 128
    edge, chunk = chosen(sum(counts) + 3, len(counts), dim, cols)
    assert edge == 128 and chunk > SEGMENT
    check(counts, 3, 1, dim, cols, [name], sum(counts))


@pytest.mark.parametrize("dim,cols,experts", [(130, 130, 128), (2000, 3, 40)])
def test_small_tiles_of_long_experts(dim, cols, experts):
    """Not in parts, as the tiles alone fill the chip: whole packs, ends inside one, and rows shorter than one."""
    counts = [SEGMENT - 40 + 3 * e % 200 for e in range(experts)]
    assert chosen(sum(counts), experts, dim, cols) == (128, None) and max(counts) > SEGMENT
    check(counts, 0, 1, dim, cols, ["f32", "bf16", "f16"], experts)
