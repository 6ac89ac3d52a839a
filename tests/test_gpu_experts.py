"""Tokens sorted by expert and back: the plan against counting pair by pair, the copies bit by bit, the weighted sums
and their gradient within bounds that count float32 roundings."""
import pytest
import torch

import train_util as tu
from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def random_ids(T, K, E, seed, dropped=0.1):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    ids[torch.rand(T, K, generator=g) < dropped] = -1
    return ids


def check_plan(ids, E):
    got = binding.gs_expert_plan(ids.cuda(), E)
    want = tu.expert_plan(ids, E)
    for name, g, w in zip(("offsets", "rows", "pairs"), (got.offsets, got.rows, got.pairs), want):
        assert torch.equal(g.cpu(), w), name
    return got, want


# around a wave, a workgroup's step and chunk, several chunks; experts from one to the most
@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (1, 8, 8), (3, 2, 5), (63, 1, 7), (64, 1, 64), (65, 1, 2), (1023, 1, 60),
                                   (1025, 1, 3), (4096, 1, 16), (4097, 1, 16), (1501, 3, 60), (8192, 8, 64),
                                   (30000, 4, 256), (500, 6, 1000), (5000, 2, 1025), (700, 3, 4096), (9000, 2, 4095)])
def test_plan(T, K, E):
    check_plan(random_ids(T, K, E, T + K + E), E)


def test_plan_of_uneven_ids():
    """All pairs to one expert, none kept, one kept, and ids past either end."""
    for E in (1, 5, 64):
        check_plan(torch.full((5000, 2), E - 1, dtype=torch.int32), E)
        check_plan(torch.full((5000, 2), -1, dtype=torch.int32), E)
        one = torch.full((5000, 2), E, dtype=torch.int32)
        check_plan(one, E)
        one[4999, 1] = 0
        check_plan(one, E)
        g = torch.Generator().manual_seed(E)
        check_plan(torch.randint(-(1 << 31), (1 << 31) - 1, (3000, 1), generator=g).to(torch.int32), E)
        check_plan(torch.arange(6000, dtype=torch.int32).remainder(E + 2).sub(1).view(-1, 3), E)


def test_plan_of_many_pairs():
    """More pairs than 256 workgroups' smallest chunks: against a stable sort."""
    T, K, E = 700001, 3, 129
    ids = random_ids(T, K, E, 3)
    got = binding.gs_expert_plan(ids.cuda(), E)
    flat = ids.reshape(-1)
    key = torch.where(flat >= 0, flat, E)
    order = torch.sort(key, stable=True).indices
    kept = int((flat >= 0).sum())
    pairs = order.to(torch.int32)
    pairs[kept:] = -1
    rows = torch.full((T * K,), -1, dtype=torch.int32)
    rows[order[:kept]] = torch.arange(kept, dtype=torch.int32)
    assert torch.equal(got.pairs.cpu(), pairs) and torch.equal(got.rows.cpu().view(-1), rows)
    assert torch.equal(got.offsets.cpu(), torch.cat([torch.zeros(1, dtype=torch.int64),
                                                     torch.bincount(key, minlength=E + 1)[:E].cumsum(0)]).int())


def test_plan_of_no_tokens():
    got = binding.gs_expert_plan(torch.zeros(0, 3, dtype=torch.int32, device="cuda"), 9)
    assert torch.equal(got.offsets.cpu(), torch.zeros(10, dtype=torch.int32)) and got.pairs.numel() == 0
    x = torch.zeros(0, 16, device="cuda")
    assert binding.gs_expert_dispatch(x, got).shape == (0, 16)
    assert binding.gs_expert_combine(x, got).shape == (0, 16)
    r = binding.gs_expert_combine_bwd(x, got, torch.zeros(0, 3, device="cuda"), x)
    assert r.rows.shape == (0, 16) and r.weights.shape == (0, 3)


def rows_inputs(T, K, E, D, dtype, seed, dropped):
    g = torch.Generator().manual_seed(seed)
    ids = random_ids(T, K, E, seed, dropped)
    x, src, gy = (torch.randn(n, D, generator=g).to(dtype) for n in (T, T * K, T))
    return ids, x, src, gy, torch.rand(T, K, generator=g)


def check_rows(ids, x, src, gy, w, E, place=lambda t: t.cuda()):
    T, K = ids.shape
    plan, (_, rows, pairs) = check_plan(ids, E)
    dx, dsrc, dgy = place(x), place(src), place(gy)
    sent = binding.gs_expert_dispatch(dx, plan, out=place(torch.full_like(src, 7)))
    assert torch.equal(sent.cpu(), tu.expert_dispatch(x, pairs, K))
    for weights in (w, None):
        y = binding.gs_expert_combine(dsrc, plan, None if weights is None else weights.cuda())
        tu.assert_within(y, tu.expert_combine(src, rows, weights)[0], tu.expert_combine_bound(src, rows, weights), "y")
    got = binding.gs_expert_combine_bwd(dsrc, plan, w.cuda(), dgy,
                                        out=binding.ExpertCombineGrad(place(torch.full_like(src, 7)),
                                                                      torch.full_like(w, 7).cuda()))
    gs, gw, size = tu.expert_combine_grad(src, rows, w, gy)
    tu.assert_within(got.rows, gs, tu.rounding(gs, src.dtype), "grad rows")
    # a lane's chain of at most D / 64 + 8 terms, 6 additions across the wave
    tu.assert_within(got.weights, gw, (x.shape[1] / 64 + 16) * tu.U * size + 1e-300, "grad weights")


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,K,E,D,dropped", [
    (1, 1, 1, 1, 0.0), (2, 3, 4, 5, 0.5), (16, 2, 8, 1024, 0.0), (50, 8, 64, 512, 0.1), (77, 3, 60, 769, 0.1),
    (33, 2, 4, 2048, 0.0), (21, 4, 16, 4096, 0.3), (9, 2, 4, 4099, 0.2), (5, 3, 4, 9001, 0.0), (700, 1, 5, 64, 0.0),
    (40, 16, 32, 130, 0.1), (300, 8, 8, 257, 1.0)])
def test_rows(T, K, E, D, dropped, name):
    check_rows(*rows_inputs(T, K, E, D, tu.DTYPES[name], T + D, dropped), E)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_rows_at_any_alignment(name):
    def place(t):
        flat = torch.zeros(t.numel() + 3, dtype=t.dtype, device="cuda")
        flat[3:] = t.reshape(-1).cuda()
        return flat[3:].view(t.shape)
    for D in (1000, 1001):
        check_rows(*rows_inputs(30, 3, 7, D, tu.DTYPES[name], D, 0.2), 7, place)


def test_dropped_pairs_and_spare_rows_are_not_read():
    """NaN in dropped pairs' weights and in the rows past the kept ones reaches no output; one in a kept row reaches
    its token alone; the bits of a row (NaN, infinities, negative zero) are copied as they are."""
    T, K, E, D = 200, 2, 6, 96
    ids, x, src, gy, w = rows_inputs(T, K, E, D, torch.float32, 5, 0.3)
    plan, (offsets, rows, pairs) = check_plan(ids, E)
    kept = int(offsets[-1])
    src[kept:] = float("nan")
    w[ids < 0] = float("nan")
    y = binding.gs_expert_combine(src.cuda(), plan, w.cuda())
    assert y.isfinite().all()
    g = binding.gs_expert_combine_bwd(src.cuda(), plan, w.cuda(), gy.cuda())
    assert g.rows.isfinite().all() and g.weights.isfinite().all()
    assert not g.rows[kept:].any() and not g.weights.cpu()[ids < 0].any()
    src[0] = float("inf")
    y = binding.gs_expert_combine(src.cuda(), plan, w.cuda()).cpu()
    token = int(pairs[0]) // K
    assert not y[token].isfinite().any() and y[[t for t in range(T) if t != token]].isfinite().all()
    x[3, :4] = torch.tensor([float("nan"), float("inf"), -0.0, 1e-45])
    sent = binding.gs_expert_dispatch(x.cuda(), plan).cpu()
    want = tu.expert_dispatch(x, pairs, K)
    assert torch.equal(sent.view(torch.int32), want.view(torch.int32))


def test_rows_of_a_plan_that_leave_the_output_are_skipped():
    """A plan's row numbers are checked by the kernels: one outside the sorted rows counts as dropped."""
    T, K, E, D = 40, 2, 4, 33
    ids, x, src, gy, w = rows_inputs(T, K, E, D, torch.float32, 6, 0.0)
    plan, (_, rows, _) = check_plan(ids, E)
    rows[5, 1], rows[6, 0], rows[7, 0] = T * K, 1 << 30, -5
    bad = binding.ExpertPlan(plan.offsets, rows.cuda(), plan.pairs)
    rows = torch.where((rows >= 0) & (rows < T * K), rows, -1)
    y = binding.gs_expert_combine(src.cuda(), bad, w.cuda())
    tu.assert_within(y, tu.expert_combine(src, rows, w)[0], tu.expert_combine_bound(src, rows, w), "y")
    g = binding.gs_expert_combine_bwd(src.cuda(), bad, w.cuda(), gy.cuda())
    assert not g.weights[5, 1].item() and not g.weights[6, 0].item() and not g.weights[7, 0].item()
    binding.gs_expert_dispatch(x.cuda(), bad)
    torch.cuda.synchronize()


def test_gradients_against_differences():
    """Combine and dispatch are linear in their rows: the gradients' products with directions are differences."""
    T, K, E, D = 60, 3, 5, 70
    ids, x, src, gy, w = rows_inputs(T, K, E, D, torch.float32, 8, 0.2)
    plan, (_, rows, pairs) = check_plan(ids, E)
    g = binding.gs_expert_combine_bwd(src.cuda(), plan, w.cuda(), gy.cuda())
    gen = torch.Generator().manual_seed(9)
    loss = lambda s, v: (gy.double() * tu.expert_combine(s, rows, v)[0]).sum().item()  # noqa: E731
    for got, at in ((g.rows, 0), (g.weights, 1)):
        args = [src.double(), w.double()]
        d = torch.randn(args[at].shape, generator=gen, dtype=torch.float64)
        up, down = [a.clone() for a in args], [a.clone() for a in args]
        up[at] += d
        down[at] -= d
        got = got.cpu().double()
        # each entry of the gradient is off by at most (2 + 16) roundings of its terms
        room = 18 * 2.0 ** -24 * (got * d).abs().sum().item() + 2.0 ** -19 * d.abs().sum().item()
        assert abs((got * d).sum().item() - (loss(*up) - loss(*down)) / 2) <= room
    gr = torch.randn(T * K, D, generator=gen)
    gx = binding.gs_expert_combine(gr.cuda(), plan).cpu().double()
    d = torch.randn(T, D, generator=gen, dtype=torch.float64)
    want = (gr.double() * tu.expert_dispatch(d, pairs, K)).sum().item()
    assert abs((gx * d).sum().item() - want) <= 4 * 2.0 ** -24 * 3 * (gx * d).abs().sum().item() + 1e-3


def test_same_bits_on_a_side_stream_and_in_a_graph():
    T, K, E, D = 3000, 4, 24, 320
    ids, x, src, gy, w = (t.cuda() for t in rows_inputs(T, K, E, D, torch.bfloat16, 11, 0.1))

    def everything(stream=None):
        plan = binding.gs_expert_plan(ids, E, stream=stream)
        g = binding.gs_expert_combine_bwd(src, plan, w, gy, stream=stream)
        return [plan.offsets, plan.rows, plan.pairs, binding.gs_expert_dispatch(x, plan, stream=stream),
                binding.gs_expert_combine(src, plan, w, stream=stream), g.rows, g.weights]
    want = everything()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = everything(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = everything()
    for k in range(3):
        ids.copy_(ids.roll(7 + k, 0))
        want = everything()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_more_elements_than_32_bits_count():
    T, K, E, D = 1 << 17, 4, 8, 4104
    ids = torch.arange(T * K, dtype=torch.int32).remainder(E).view(T, K)
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    plan = binding.gs_expert_plan(ids.cuda(), E)
    sent = binding.gs_expert_dispatch(x, plan)
    last = plan.pairs[-50:].long() // K
    assert torch.equal(sent[-50:], x[last])
    y = binding.gs_expert_combine(sent, plan)
    # four equal rows: the sum is four times the row, exactly
    assert torch.equal(y[-100:], x[-100:] * 4)
    g = binding.gs_expert_combine_bwd(sent, plan, torch.full((T, K), 0.5, device="cuda"), x)
    assert torch.equal(g.rows[-50:], x[last] * 0.5)


@pytest.mark.parametrize("T,K,E", [(4097, 64, 7), (200001, 2, 33), (150000, 3, 2000), (270000, 1, 1)])
def test_plan_of_more_pairs_than_a_step_of_every_workgroup(T, K, E):
    check_plan(random_ids(T, K, E, T + K + E), E)
