"""The router and the 8-bit operators at the ends of what they take: plans that are no plan's, long rows, captured calls,
other streams, calls side by side, outputs and workspaces of the caller."""
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


def held(*shape, seed=0):
    return binding.gs_quantize(torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda())


@pytest.mark.parametrize("seed", range(4))
def test_a_plan_of_garbage_stays_in_bounds(seed):
    """Offsets and pairs out of range, in no order: the rows' numbers are taken to their ends, and what lies around the
    outputs stays as it was."""
    T, K, E, D, N = 150, 2, 5, 200, 136
    g = torch.Generator().manual_seed(seed)
    plan = binding.ExpertPlan(torch.randint(-400, 800, (E + 1,), generator=g, dtype=torch.int32).cuda(),
                              torch.zeros(T, K, dtype=torch.int32, device="cuda"),
                              torch.randint(-1000, 1000, (T * K,), generator=g, dtype=torch.int32).cuda())
    x, w = held(T, D, seed=seed), held(E, N, D, seed=seed)
    for dtype in (torch.float32, torch.bfloat16):
        around = torch.full((T * K + 20, N), 7.0, dtype=dtype, device="cuda")
        binding.gs_expert_product(x, w, plan, gather=True, dtype=dtype, out=around[10:-10])
        assert (around[:10] == 7).all() and (around[-10:] == 7).all()
    grad = torch.randn(T * K, N, generator=g).cuda()
    around = torch.full((E + 2, D, N), 7.0, device="cuda")
    binding.gs_expert_weight_grad(x, grad, plan, gather=True, out=around[1:-1])
    assert (around[0] == 7).all() and (around[-1] == 7).all()


def test_parts_of_garbage_stay_in_bounds():
    """The same where the sums are made in parts, whose number the offsets give."""
    T, E, D, N = 9000, 6, 64, 40
    g = torch.Generator().manual_seed(1)
    x, grad = held(T, D), torch.randn(T, N, generator=g).cuda()
    need = binding.load_library().gs_expert_weight_grad_workspace_bytes(T, E, D, N)
    assert need > 0
    for seed in range(3):
        off = torch.randint(0, T + 1, (E + 1,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
        off[::2] = 0
        off[1::2] = T  # every second expert has all rows: more parts than there is room for
        plan = binding.ExpertPlan(off.cuda(), torch.zeros(T, 1, dtype=torch.int32, device="cuda"),
                                  torch.arange(T, dtype=torch.int32, device="cuda"))
        room = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
        binding.gs_expert_weight_grad(x, grad, plan, workspace=room[256:-256])
        assert (room[:256] == 7).all() and (room[-256:] == 7).all()


def test_long_rows():
    """More blocks than scales are held at once, in the largest tiles and the smaller ones; whole numbers, so exact."""
    g = torch.Generator().manual_seed(4)
    D = 128 * 70 + 5
    w = torch.randint(-3, 4, (300, D), generator=g).float()
    qw = binding.gs_quantize(w.cuda())
    for R in (40, 20000):
        x = torch.randint(-3, 4, (R, D), generator=g).float()
        got = binding.gs_expert_product(binding.gs_quantize(x.cuda()), qw, dtype=torch.float16)
        pick = torch.arange(0, R, max(1, R // 50))
        assert torch.equal(got.cpu()[pick], (x[pick].double() @ w.double().T).to(torch.float16))


@pytest.mark.parametrize("D", [256, 1024])
def test_the_largest_tiles_with_odd_ends(D):
    """Rows and columns that end inside the largest tiles, an expert of one row and one without any."""
    g = torch.Generator().manual_seed(D)
    counts = [3001, 1, 0, 2600, 3007]
    E, N = len(counts), 1029
    off = torch.tensor([0] + counts).cumsum(0).int()
    T = int(off[-1]) + 77
    plan = binding.ExpertPlan(off.cuda(), torch.zeros(T, 1, dtype=torch.int32, device="cuda"),
                              torch.arange(T, dtype=torch.int32, device="cuda"))
    x = torch.randint(-4, 5, (T, D), generator=g).float()
    w = torch.randint(-4, 5, (E, N, D), generator=g).float()
    grad = torch.randint(-4, 5, (T, N), generator=g).to(torch.bfloat16)
    qx, qw = binding.gs_quantize(x.cuda()), binding.gs_quantize(w.cuda())
    got = binding.gs_expert_product(qx, qw, plan, dtype=torch.float16).cpu()
    for e in range(E):
        of = slice(int(off[e]), int(off[e + 1]))
        assert torch.equal(got[of], (x[of] @ w[e].T).to(torch.float16))  # below 2^24: exact in float32 too
    assert (got[int(off[-1]):] == 0).all()
    got = binding.gs_expert_weight_grad(qx, grad.cuda(), plan).cpu()
    for e in range(E):
        of = slice(int(off[e]), int(off[e + 1]))
        assert torch.equal(got[e], x[of].T @ grad[of].float())


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_weight_grad_of_large_tiles(name):
    """Matrices that fill the chip by themselves: the largest tiles in every type, columns that end inside a pack too."""
    g = torch.Generator().manual_seed(6)
    E, D, T = 40, 1000, 2500
    ids = torch.randint(-1, E, (T, 1), generator=g, dtype=torch.int32)
    off, _, pairs = tu.expert_plan(ids, E)
    plan = binding.gs_expert_plan(ids.cuda(), E)
    x = torch.randint(-7, 8, (T, D), generator=g).float()
    qx = binding.gs_quantize(x.cuda())
    rows = fu.sorted_rows(x, pairs, 1)
    for N in (1000, 1003):
        grad = torch.randint(-7, 8, (T, N), generator=g).to(tu.DTYPES[name])
        got = binding.gs_expert_weight_grad(qx, grad.cuda(), plan, gather=True).cpu()
        for e in range(E):
            of = slice(int(off[e]), int(off[e + 1]))
            assert torch.equal(got[e], rows[of].T @ grad[of].float()), e


def test_captured_calls():
    """Every operator in one graph; replays with new inputs and eager work between give what eager calls give."""
    T, K, E, D, N = 700, 2, 6, 200, 136
    g = torch.Generator().manual_seed(7)
    logits = [torch.randn(T, E, generator=g).cuda() for _ in range(3)]
    xs = [torch.randn(T, D, generator=g).cuda() for _ in range(3)]
    qw = held(E, N, D, seed=8)
    gw, gl = torch.randn(T, K, generator=g).cuda(), torch.full((), 0.1, device="cuda")

    def calls(logit, x):
        route = binding.gs_expert_route(logit, K)
        plan = binding.gs_expert_plan(route.ids, E)
        q = binding.gs_quantize(x)
        y = binding.gs_expert_product(q, qw, plan, gather=True, relu=True)
        return [route.weights, route.counts, route.loss, binding.gs_expert_route_bwd(logit, route, gw, gl),
                binding.gs_dequantize(q), y, binding.gs_expert_weight_grad(q, y, plan, gather=True),
                binding.gs_quantize(x, transpose=True).values.view(torch.uint8)]
    logit, x = logits[0].clone(), xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(logit, x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(logit, x)
    for k in (0, 1, 2, 1, 0):
        logit.copy_(logits[k])
        x.copy_(xs[k])
        graph.replay()
        want = calls(logits[k], xs[k])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_streams_side_by_side():
    """The same calls on two streams at once, each with the workspaces that it allocates."""
    T, E, D, N = 30000, 8, 128, 64
    g = torch.Generator().manual_seed(9)
    logits, grad = torch.randn(T, E, generator=g).cuda(), torch.randn(T, N, generator=g).cuda()
    x = held(T, D, seed=1)
    want = binding.gs_expert_route(logits, 2), binding.gs_expert_weight_grad(x, grad)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s in streams:
            got.append((binding.gs_expert_route(logits, 2, stream=s), binding.gs_expert_weight_grad(x, grad, stream=s)))
    torch.cuda.synchronize()
    for route, weight in got:
        assert torch.equal(route.ids, want[0].ids) and torch.equal(route.shares, want[0].shares)
        assert torch.equal(route.loss, want[0].loss) and torch.equal(weight, want[1])


def test_outputs_and_workspaces_of_the_caller():
    lib = binding.load_library()
    logits = torch.randn(20000, 70, device="cuda")
    want = binding.gs_expert_route(logits, 3)
    out = binding.ExpertRoute(*(torch.full_like(t, 7) for t in (want.ids, want.weights, want.counts, want.shares,
                                                                want.loss, want.kept)))
    ws = torch.empty(lib.gs_expert_route_workspace_bytes(20000, 70), dtype=torch.uint8, device="cuda")
    got = binding.gs_expert_route(logits, 3, out=out, workspace=ws)
    assert got is out
    for a, b in ((got.ids, want.ids), (got.weights, want.weights), (got.counts, want.counts),
                 (got.shares, want.shares), (got.loss, want.loss), (got.kept, want.kept)):
        assert torch.equal(a, b)
    with pytest.raises(binding.GsError, match="workspace"):
        binding.gs_expert_route(logits, 3, workspace=ws[:-1])
    x = torch.randn(5, 300, device="cuda")
    q = binding.gs_quantize(x)
    into = binding.Quantized(torch.empty_like(q.values), torch.empty_like(q.scales), 300)
    assert binding.gs_quantize(x, out=into) is into and torch.equal(into.scales, q.scales)
    with pytest.raises(ValueError, match="out must hold"):
        binding.gs_quantize(x[:4].contiguous(), out=into)
    with pytest.raises(ValueError, match="rows"):
        binding.gs_expert_product(q, held(8, 300), binding.gs_expert_plan(torch.zeros(5, 2, dtype=torch.int32,
                                                                                      device="cuda"), 1))
    with pytest.raises(ValueError, match="weight must hold"):
        binding.gs_expert_product(q, held(8, 301))


def test_a_product_of_no_rows():
    plan = binding.gs_expert_plan(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 3)
    x = binding.gs_quantize(torch.zeros(0, 40, device="cuda"))
    assert binding.gs_expert_product(x, held(3, 7, 40), plan, gather=True).shape == (0, 7)
    got = binding.gs_expert_weight_grad(x, torch.zeros(0, 7, device="cuda"), plan, gather=True,
                                        out=torch.full((3, 40, 7), 5.0, device="cuda"))
    assert (got == 0).all()
