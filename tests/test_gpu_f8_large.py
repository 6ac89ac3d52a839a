"""The product's largest tiles, which long sums of many rows take: ends inside a tile, an expert of one row, one without
any, rows past the kept ones, and more blocks than scales are held at once. Whole numbers, so every sum is exact."""
import pytest
import torch

from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("D,dtype", [(2100, torch.float16), (2048, torch.bfloat16), (4300, torch.float16)])
def test_largest_tiles(D, dtype):
    g = torch.Generator().manual_seed(D)
    counts = [6001, 1, 0, 4600, 6107]
    E, N = len(counts), 1029
    off = torch.tensor([0] + counts).cumsum(0).int()
    T = int(off[-1]) + 77
    assert T // E >= 512 and T // 256 * -(-N // 256) >= 256  # what the largest tiles take
    source = torch.randperm(T, generator=g).to(torch.int32)
    plan = binding.ExpertPlan(off.cuda(), torch.zeros(T, 1, dtype=torch.int32, device="cuda"), source.cuda())
    x = torch.randint(-3, 4, (T, D), generator=g).float()
    w = torch.randint(-3, 4, (E, N, D), generator=g).float()
    qx, qw = binding.gs_quantize(x.cuda()), binding.gs_quantize(w.cuda())
    for relu in (False, True):
        around = torch.full((T + 2, N), 7.0, dtype=dtype, device="cuda")
        binding.gs_expert_product(qx, qw, plan, gather=True, relu=relu, dtype=dtype, out=around[1:-1])
        got = around.cpu()
        assert (got[0] == 7).all() and (got[-1] == 7).all()
        got = got[1:-1]
        assert (got[int(off[-1]):] == 0).all()
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            # each tile's first and last rows and some between
            pick = [r for r in range(lo, hi) if (r - lo) % 256 in (0, 1, 31, 130, 255) or r == hi - 1]
            if pick:
                want = x[source[pick].long()] @ w[e].T
                assert torch.equal(got[pick], (want.clamp(min=0) if relu else want).to(dtype)), (e, relu)
