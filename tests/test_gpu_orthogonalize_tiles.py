"""Orthogonalised updates of large matrices and stacks, whose products take tiles of 128, 192 and 256: entry by entry
against the steps in 64 bits on the device, and the same bits again."""
import os
import re

import pytest
import torch

import train_util as tu
from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding
from test_gpu_orthogonalize_accuracy import matrix

pytestmark = pytest.mark.gpu
SOURCE = os.path.join(os.path.dirname(binding.__file__), "csrc", "ortho.hip")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def tiles(batch, m, n):
    """The tile edges of a step's three products, by the library's rule with the costs that stand in its source."""
    with open(SOURCE) as f:
        row = re.search(r"edges\[\] = \{(.*)\};", f.read()).group(1)
    costs = [(int(e), float(c)) for e, c in re.findall(r"\{(\d+), ([\d.]+)\}", row)]
    assert sorted(e for e, _ in costs) == [64, 128, 192, 256]
    M, N = (-(-v // 32) * 32 for v in sorted((m, n)))

    def edge(rows, cols, symmetric):
        def cost(of):
            e, c = of
            r, k = -(-rows // e), -(-cols // e)
            count = batch * (r * (r + 1) // 2 if symmetric else r * k)
            return -(-count // 256) * e * e * c
        return min(costs, key=cost)[0]
    return {edge(M, M, True), edge(M, N, False)}


CASES = [((4096, 4096), "f32"), ((4096, 4096), "bf16"), ((4090, 3999), "f16"), ((3999, 4090), "f32"),
         ((8, 1000, 1050), "f32"), ((8, 1050, 1000), "f16"), ((2, 2000, 1900), "bf16"), ((20, 700, 800), "f16"),
         ((20, 800, 700), "f32"), ((1600, 8000), "f32"), ((16, 500, 512), "bf16")]


def stack(shape, dtype):
    batch = shape[0] if len(shape) == 3 else 1
    u = torch.stack([matrix("momentum", *shape[-2:], seed=i) * 4.0 ** (i % 4) for i in range(batch)])
    return u.to(dtype).view(shape)


def test_every_tile_is_among_the_cases():
    for length in (2, 3):
        used = set()
        for shape, _ in CASES:
            if len(shape) == length:
                used |= tiles(shape[0] if length == 3 else 1, *shape[-2:])
        assert used >= {192, 256}, (length, used)
    assert {128} <= tiles(16, 500, 512)


@pytest.mark.parametrize("shape,name", CASES)
def test_entry_by_entry(shape, name):
    """The bound: four times what the steps in 64 bits are off by with random roundings of 22 bits in every operand, the
    worst of three runs, and the rounding of the result."""
    dtype = tu.DTYPES[name]
    u = stack(shape, dtype)
    got = binding.gs_orthogonalize(u)
    ms, gots = u.view(-1, *shape[-2:]), got.view(-1, *shape[-2:])
    for i in sorted({0, 1, len(ms) // 2, len(ms) - 1} & set(range(len(ms)))):
        with torch.device("cuda"):
            want = tu.orthogonalize(ms[i])
            worst = 0.0
            for k in range(3):
                g = torch.Generator(device="cuda").manual_seed(k)
                worst = max(worst, (tu.orthogonalize(ms[i].float(), noise=g) - want).abs().max().item())
            off = (gots[i].double() - want).abs() - (4 * worst + tu.rounding(want, dtype))
        assert not gots[i].isnan().any() and off.max().item() <= 0, \
            f"matrix {i}: {int((off > 0).sum())} entries beyond the bound, worst by {off.max().item():.3g}"
        own = (want.to(dtype).double() - want).norm().item()
        assert dtype == torch.float32 or (gots[i].double() - want).norm().item() <= 1.02 * own
    room = binding.load_library().gs_orthogonalize_workspace_bytes(len(ms), *shape[-2:])
    ws = torch.full((room,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(binding.gs_orthogonalize(u, workspace=ws), got)


@pytest.mark.parametrize("shape", [(8, 1000, 1050), (20, 800, 700)])
def test_in_a_graph(shape):
    u = stack(shape, torch.float16)
    first = u.clone()
    binding.gs_orthogonalize(u)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = binding.gs_orthogonalize(u)
    for k in range(3):
        u.copy_(first.roll(k, 0))
        want = binding.gs_orthogonalize(u)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want)
