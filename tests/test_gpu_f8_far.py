"""The router and the 8-bit operators where offsets pass 2^32 elements, and layers of no tokens."""
import pytest
import torch

from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding
from tile_binned_gaussian_amd.expert_layer import ExpertLayer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def test_router_of_many_logits():
    """The same 997 rows over and over, 2^32 logits and some."""
    E, K, n = 256, 2, (1 << 24) + 5
    rows = torch.randn(997, E, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    logits = rows[torch.arange(n, device="cuda") % 997]
    assert logits.numel() > 1 << 32
    few, many = binding.gs_expert_route(rows, K), binding.gs_expert_route(logits, K)
    at = torch.arange(n, device="cuda") % 997
    assert torch.equal(many.ids, few.ids[at]) and torch.equal(many.weights, few.weights[at])
    assert torch.equal(many.counts, torch.bincount(many.ids.reshape(-1).long(), minlength=E).int())
    gw = torch.randn(997, K, generator=torch.Generator().manual_seed(2)).cuda()
    got = binding.gs_expert_route_bwd(logits, many, gw[at].contiguous())
    want = binding.gs_expert_route_bwd(rows, few, gw)
    for first in range(0, n, 1 << 21):
        assert torch.equal(got[first:first + (1 << 21)], want[at[first:first + (1 << 21)]])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_held_rows_products_and_gradients(dtype):
    """Rows of whole numbers, every 1009 of them the same."""
    R, D, N, period = 1100001, 300, 4100, 1009
    g = torch.Generator().manual_seed(3)
    x, w = (torch.randint(-3, 4, shape, generator=g).float() for shape in ((period, D), (N, D)))
    at = torch.arange(R, device="cuda") % period
    q = binding.gs_quantize(x.cuda()[at].to(dtype))
    few = binding.gs_quantize(x.cuda())
    qw = binding.gs_quantize(w.cuda())
    got = binding.gs_expert_product(q, qw, dtype=dtype)
    assert got.numel() > 1 << 32
    want = binding.gs_expert_product(few, qw, dtype=dtype)
    assert torch.equal(want.cpu(), (x @ w.T).to(dtype))
    for first in range(0, R, 1 << 17):
        assert torch.equal(got[first:first + (1 << 17)], want[at[first:first + (1 << 17)]]), first
    # the gradient of rows that are zero but for some of the last ones
    got.zero_()
    some = torch.randint(-3, 4, (100, N), generator=g).to(dtype).cuda()
    got[-100:] = some
    grad = binding.gs_expert_weight_grad(q, got).cpu()
    assert torch.equal(grad, x[at[-100:].cpu()].T @ some.cpu().float())


def test_held_values_past_2_32():
    R, D, period = 4200001, 1040, 1013
    x = torch.randn(period, D, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    at = torch.arange(R, device="cuda") % period
    q, few = binding.gs_quantize(x[at]), binding.gs_quantize(x)
    assert q.values.numel() > 1 << 32
    want = few.values.view(torch.uint8)
    back, short = binding.gs_dequantize(q, dtype=torch.bfloat16), binding.gs_dequantize(few, dtype=torch.bfloat16)
    for first in range(0, R, 1 << 19):
        of = at[first:first + (1 << 19)]
        assert torch.equal(q.values.view(torch.uint8)[first:first + (1 << 19)], want[of]), first
        assert torch.equal(q.scales[first:first + (1 << 19)], few.scales[of])
        assert torch.equal(back[first:first + (1 << 19)], short[of])


@pytest.mark.parametrize("products,balance", [("library", 0.0), ("library", 0.1), ("f8", 0.0), ("f8", 0.1)])
def test_a_layer_of_no_tokens(products, balance):
    layer = ExpertLayer(24, 16, 4, 2, products=products, balance=balance)
    x = torch.zeros(0, 24, dtype=torch.bfloat16, device="cuda")
    y, saved = layer.forward(x)
    grad_x, grads = layer.backward(saved, x)
    assert y.shape == grad_x.shape == (0, 24)
    for name, p in layer.parameters.items():
        assert grads[name].shape == p.shape and (grads[name] == 0).all(), name
