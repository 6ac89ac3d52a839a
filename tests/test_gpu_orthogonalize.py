"""Orthogonalised updates against the Newton-Schulz steps in 64 bits, within what the same steps are off by with
random roundings of the kernels' sizes."""
import pytest
import torch

import train_util as tu
from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def momentum(shape, dtype, seed=0):
    """A few strong directions and a bulk of weak ones."""
    g = torch.Generator().manual_seed(seed)
    m, n = shape[-2:]
    r = max(1, min(m, n) // 32)
    u = torch.randn(*shape[:-1], r, generator=g) @ torch.randn(*shape[:-2], r, n, generator=g)
    return (u * (1e-3 / r ** 0.5) + 3e-4 * torch.randn(*shape, generator=g)).to(dtype)


def check(u, got, **kw):
    want = tu.orthogonalize(u, **kw)
    entry, norm = tu.orthogonalize_bound(u, want, **kw)
    tu.assert_within(got, want, entry, "out")
    off = (got.cpu().double() - want).norm().item()
    assert off <= norm, f"2-norm of the error {off:.3g} beyond {norm:.3g}"


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 50), (7, 3), (32, 32), (63, 65), (64, 64), (96, 160), (129, 128),
                                 (160, 96), (200, 513), (300, 1000), (777, 333), (640, 640), (1025, 130), (33, 4000),
                                 (780, 900)])
def test_one_matrix(m, n, name):
    u = momentum((m, n), tu.DTYPES[name], m + n)
    check(u, binding.gs_orthogonalize(u.cuda()))


@pytest.mark.parametrize("shape", [(3, 40, 70), (5, 130, 64), (2, 300, 260), (16, 96, 160)])
def test_a_batch(shape):
    for dtype in tu.DTYPES.values():
        u = momentum(shape, dtype, 4)
        u[1] *= 64.0  # each matrix has its own norm
        got = binding.gs_orthogonalize(u.cuda())
        for i in range(shape[0]):
            check(u[i], got[i])


def test_other_steps_and_coefficients():
    u = momentum((100, 140), torch.float32, 1)
    cubic = (1.5, -0.5, 0.0)
    for steps, kw in ((0, {}), (1, {}), (2, {}), (9, {}), (12, {"coefficients": cubic}), (3, {"eps": 1e-2})):
        check(u, binding.gs_orthogonalize(u.cuda(), steps=steps, **kw), steps=steps, **kw)
        h = u.bfloat16()
        check(h, binding.gs_orthogonalize(h.cuda(), steps=steps, **kw), steps=steps, **kw)


def test_matrices_of_no_size_and_of_no_scale():
    """Zeros give zeros; a batch of none; entries whose squares leave float32's range either way."""
    zero = torch.zeros(2, 50, 60, device="cuda")
    assert not binding.gs_orthogonalize(zero).any()
    assert binding.gs_orthogonalize(torch.zeros(0, 50, 60, device="cuda")).shape == (0, 50, 60)
    for scale in (1e30, 1e-30):
        u = momentum((70, 90), torch.float32, 2) * scale
        check(u, binding.gs_orthogonalize(u.cuda(), eps=0.0), eps=0.0)


def test_a_matrix_that_is_not_finite_spoils_no_other():
    for bad in (float("nan"), float("inf")):
        for m, n in ((60, 80), (300, 200)):
            u = momentum((3, m, n), torch.float32, 3)
            want = binding.gs_orthogonalize(u.cuda())
            u[1, 5, 7] = bad
            got = binding.gs_orthogonalize(u.cuda())
            assert got[1].isnan().all()
            assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


def test_rank_one_and_repeated_rows():
    g = torch.Generator().manual_seed(5)
    u = torch.randn(130, 1, generator=g) @ torch.randn(1, 90, generator=g)
    left, _, right = torch.linalg.svd(u.double(), full_matrices=False)
    a, b, c = tu.COEFFICIENTS
    s = 1.0
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    got = binding.gs_orthogonalize(u.cuda()).cpu().double()
    # directions that are rounding alone (2^-22 of the entries in any of 6 roundings a step) grow by at most 3.45 a
    # step: 490 in five steps, of a matrix whose 2-norm is 1
    assert (got - s * left[:, :1] @ right[:1]).norm().item() <= 6 * 490 * 2.0 ** -22


def test_in_place_and_at_any_alignment():
    for dtype in tu.DTYPES.values():
        u = momentum((150, 201), dtype, 6)
        want = binding.gs_orthogonalize(u.cuda())
        flat = torch.zeros(u.numel() + 11, dtype=dtype, device="cuda")
        inside = flat[3:3 + u.numel()].view(u.shape)
        inside.copy_(u)
        got = binding.gs_orthogonalize(inside, out=inside)
        assert got.data_ptr() == inside.data_ptr() and torch.equal(inside, want)
        assert not flat[:3].any() and not flat[-8:].any()


def test_same_bits_on_a_side_stream_and_in_a_graph():
    for shape in ((4, 96, 128), (500, 260)):
        u = momentum(shape, torch.float32, 7).cuda()
        want = binding.gs_orthogonalize(u)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = binding.gs_orthogonalize(u, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = binding.gs_orthogonalize(u)
        for k in range(3):
            u.add_(1e-4 * k)
            want = binding.gs_orthogonalize(u)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(held, want)


def test_a_large_matrix_on_the_device():
    """2500 x 1111 and 2048 x 2048 against the steps in float64 on the GPU (library products): 2-norm only."""
    for shape, dtype, room in (((2500, 1111), torch.float32, 2.0 ** -18), ((2048, 2048), torch.bfloat16, 2.0 ** -8)):
        u = momentum(shape, dtype, 8).cuda()
        x = u.double()
        x = x / (x.norm() + 1e-7)
        x = x.T.contiguous() if shape[0] > shape[1] else x
        a, b, c = tu.COEFFICIENTS
        for _ in range(5):
            A = torch.mm(x, x.T.contiguous())
            x = a * x + torch.mm(b * A + c * torch.mm(A, A), x)
        x = x.T if shape[0] > shape[1] else x
        got = binding.gs_orthogonalize(u).double()
        # float32: 15 products of 2^-22 and less, grown by at most a few; bfloat16: the result's own 2^-9 and the
        # first steps' 2^-12, grown likewise
        assert ((got - x).norm() / x.norm()).item() <= room


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(64, 3001), (300, 4000), (4100, 200), (2, 130, 5000), (33, 20011), (500, 2100)])
def test_few_tiles_of_many_columns(shape, name):
    """Workgroups share a tile's sum: right, and the same bits again, from a workspace full of anything and in a graph."""
    u = momentum(shape, tu.DTYPES[name], sum(shape))
    d = u.cuda()
    got = binding.gs_orthogonalize(d)
    for i in range(shape[0] if len(shape) == 3 else 1):
        check(u[i], got[i]) if len(shape) == 3 else check(u, got)
    batch = shape[0] if len(shape) == 3 else 1
    room = binding.load_library().gs_orthogonalize_workspace_bytes(batch, *shape[-2:])
    ws = torch.full((room,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(binding.gs_orthogonalize(d, workspace=ws), got)
    out = torch.empty_like(d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.gs_orthogonalize(d, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        ws.fill_(170)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got)


def test_shared_tiles_with_high_halves_alone():
    u = momentum((770, 2000), torch.bfloat16, 5)
    check(u, binding.gs_orthogonalize(u.cuda()))
