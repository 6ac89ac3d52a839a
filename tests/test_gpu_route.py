"""The router: choices against passes over each row, weights, counts, shares and balance loss against 64 bits, and the
gradient against the formula."""
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


def inputs(T, E, K, name, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, E, generator=g) + 0.5 * torch.randn(E, generator=g)).to(tu.DTYPES[name])
    return x, torch.rand(T, generator=g) < 0.8, torch.randn(T, K, generator=g)


def check(x, K, mask, renormalize, gw, gl=0.3, place=lambda t: t.cuda()):
    T, E = x.shape
    got = binding.gs_expert_route(place(x), K, mask=None if mask is None else mask.cuda(), renormalize=renormalize)
    ids, w, counts, shares, loss, kept = fu.route(x, K, mask, renormalize)
    assert torch.equal(got.ids.cpu(), ids) and torch.equal(got.counts.cpu(), counts.int())
    assert got.kept.item() == kept and got.loss.shape == ()
    b_w, b_s, b_l = fu.route_bounds(x, ids, w, shares, counts, kept)
    tu.assert_within(got.weights, w, b_w, "weights")
    tu.assert_within(got.shares, shares, b_s, "shares")
    tu.assert_within(got.loss, loss, b_l, "loss")
    for g1, g2 in ((gw, gl), (gw, None), (None, gl), (None, None)):
        grad = binding.gs_expert_route_bwd(place(x), got, None if g1 is None else g1.cuda(),
                                           None if g2 is None else torch.tensor(g2, device="cuda"),
                                           renormalize=renormalize)
        want, size = fu.route_grad(x, ids, got.weights.cpu(), counts, kept, torch.zeros_like(gw) if g1 is None else g1,
                                   0.0 if g2 is None else g2, renormalize)
        assert grad.dtype == x.dtype
        tu.assert_within(grad, want, fu.route_grad_bound(x, want, size, K), "grad logits")
    return got


# around a group of lanes and a wave, one workgroup and many; experts from one to the most
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (3, 2, 2), (257, 3, 1), (16, 8, 2), (33, 7, 7), (600, 16, 2),
                                   (65, 17, 4), (100, 31, 3), (9, 64, 8), (1501, 60, 3), (40, 65, 5), (77, 128, 8),
                                   (21, 200, 6), (30, 257, 2), (12, 1000, 8), (7, 1025, 4), (5, 4096, 8),
                                   (9, 4095, 1)])
def test_route(T, E, K, name):
    x, mask, gw = inputs(T, E, K, name, T + E)
    for renormalize in (True, False):
        check(x, K, None, renormalize, gw)
        check(x, K, mask, renormalize, gw)


def test_many_tokens():
    """More tokens than one turn of all workgroups, by a stable sort."""
    T, E, K = 700001, 5, 2
    x, mask, _ = inputs(T, E, K, "bf16", 4)
    got = binding.gs_expert_route(x.cuda(), K, mask=mask.cuda())
    ids = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :K].int()
    ids[~mask] = -1
    assert torch.equal(got.ids.cpu(), ids)
    _, w, counts, shares, loss, kept = fu.route(x, K, mask, ids=ids)
    b_w, b_s, b_l = fu.route_bounds(x, ids, w, shares, counts, kept)
    assert torch.equal(got.counts.cpu(), counts.int()) and got.kept.item() == kept
    for a, b, c, what in ((got.weights, w, b_w, "weights"), (got.shares, shares, b_s, "shares"),
                          (got.loss, loss, b_l, "loss")):
        tu.assert_within(a, b, c, what)


@pytest.mark.parametrize("E", [2, 8, 60, 70, 300])
def test_equal_logits_go_to_the_lowest_index(E):
    g = torch.Generator().manual_seed(E)
    x = torch.randint(-1, 2, (200, E), generator=g).float()
    x[::3] = torch.where(x[::3] == 0, -0.0, x[::3])  # both zeros are one value
    x[1::3][:, ::2] = -0.0
    x[5] = 0
    check(x, min(E, 4), None, True, torch.randn(200, min(E, 4), generator=g))


@pytest.mark.parametrize("E,K", [(4, 3), (8, 8), (60, 5), (130, 4)])
def test_experts_that_may_not_be_chosen(E, K):
    """Logits of minus infinity, down to rows where nothing is left."""
    g = torch.Generator().manual_seed(E)
    x = torch.randn(90, E, generator=g)
    x[torch.rand(90, E, generator=g) < 0.6] = float("-inf")
    x[3] = float("-inf")
    x[4] = float("-inf")
    x[4, E - 1] = -1e30
    x[5] = torch.finfo(torch.float32).min  # the type's lowest value is a number
    mask = torch.rand(90, generator=g) < 0.9
    mask[4:6] = True
    for renormalize in (True, False):
        got = check(x, K, mask, renormalize, torch.randn(90, K, generator=g))
        assert got.ids[3].tolist() == [-1] * K and got.ids[4].tolist() == [E - 1] + [-1] * (K - 1)
        assert got.ids[5].tolist() == list(range(K))


@pytest.mark.parametrize("E", [8, 60, 130])
def test_no_number(E):
    """A NaN is chosen first, before an infinity; the row's weights, the shares and the loss say so, other rows do not."""
    x = torch.randn(50, E, generator=torch.Generator().manual_seed(E))
    x[7, 3] = float("nan")
    x[7, 5] = float("inf")
    x[9, 4] = float("inf")
    got = binding.gs_expert_route(x.cuda(), 2)
    assert got.ids[7].tolist() == [3, 5] and got.ids[9, 0].item() == 4
    bad = torch.tensor([t in (7, 9) for t in range(50)])
    assert got.weights.cpu()[bad].isnan().all() and got.weights.cpu()[~bad].isfinite().all()
    assert got.loss.isnan() and got.shares.isnan().all()
    ids = fu.choose(x.double(), 2)
    assert torch.equal(got.ids.cpu(), ids)
    # left out, they disturb nothing
    masked = binding.gs_expert_route(x.cuda(), 2, mask=~bad.cuda())
    assert masked.loss.isfinite() and masked.shares.isfinite().all() and masked.weights.isfinite().all()
    grad = binding.gs_expert_route_bwd(x.cuda(), masked, torch.ones(50, 2, device="cuda"),
                                       torch.ones((), device="cuda")).cpu()
    assert grad.isfinite().all() and (grad[bad] == 0).all()


@pytest.mark.parametrize("T", [0, 1, 300, 5000])
def test_nothing_routed(T):
    x = torch.randn(T, 70, device="cuda")
    got = binding.gs_expert_route(x, 3, mask=torch.zeros(T, dtype=torch.bool, device="cuda"))
    assert (got.ids == -1).all() and (got.weights == 0).all() and (got.counts == 0).all()
    assert (got.shares == 0).all() and got.loss.item() == 0 and got.kept.item() == 0
    grad = binding.gs_expert_route_bwd(x, got, torch.ones(T, 3, device="cuda"), torch.ones((), device="cuda"))
    assert grad.shape == (T, 70) and (grad == 0).all()


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_rows_at_any_alignment(name):
    def place(t):
        flat = torch.zeros(t.numel() + 3, dtype=t.dtype, device="cuda")
        flat[3:] = t.reshape(-1).cuda()
        return flat[3:].view(t.shape)
    for E in (5, 8, 16, 60, 131):
        x, mask, gw = inputs(70, E, 2, name, E)
        check(x, 2, mask, True, gw, place=place)


def test_large_logits():
    """Differences of hundreds: probabilities down to zero, none of them lost to an overflow."""
    x = torch.randn(64, 12, generator=torch.Generator().manual_seed(1)) * 300
    check(x, 3, None, True, torch.randn(64, 3, generator=torch.Generator().manual_seed(2)))


def test_shares_of_equal_rows():
    """2^20 rows alike: a share is the row's probability, whatever the number of rows."""
    row = torch.randn(1, 8, generator=torch.Generator().manual_seed(3))
    got = binding.gs_expert_route(row.expand(1 << 20, 8).contiguous().cuda(), 2)
    p = torch.softmax(row.double(), dim=1)[0]
    # 64 equal terms and tokens / 64 / (1024 workgroups x 32 rows) of such sums in a lane, 256 lanes
    assert ((got.shares.cpu().double() - p).abs() <= p * tu.U * (64 + 256 + 100)).all()
    best = row[0].sort(descending=True, stable=True).indices[:2]
    assert got.counts.cpu().sum() == 1 << 21 and (got.counts.cpu()[best] == 1 << 20).all()
    same = binding.gs_expert_route(row.expand(1 << 20, 8).contiguous().cuda(), 2)
    assert torch.equal(same.shares, got.shares) and torch.equal(same.loss, got.loss)
