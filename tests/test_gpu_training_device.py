"""The training operators refuse a stream of another device than their tensors' before anything is launched."""
import pytest
import torch

from gpu_util import require_gpu
from tile_binned_gaussian_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def calls():
    T, K, E, D = 6, 2, 3, 16
    x, w = torch.randn(T, D, device="cuda"), torch.ones(D, device="cuda")
    norm = binding.gs_layer_norm_fwd(x, w, w)
    logits = torch.randn(T, E, device="cuda")
    route = binding.gs_expert_route(logits, K)
    plan = binding.gs_expert_plan(route.ids, E)
    rows = binding.gs_expert_dispatch(x, plan)
    q, qw = binding.gs_quantize(x), binding.gs_quantize(torch.randn(E, 5, D, device="cuda"))
    return {
        "layer_norm_fwd": lambda **k: binding.gs_layer_norm_fwd(x, w, w, **k).y,
        "layer_norm_bwd": lambda **k: binding.gs_layer_norm_bwd(x, w, norm.mean, norm.rstd, x, **k).x,
        "expert_plan": lambda **k: binding.gs_expert_plan(route.ids, E, **k).rows,
        "expert_dispatch": lambda **k: binding.gs_expert_dispatch(x, plan, **k),
        "expert_combine": lambda **k: binding.gs_expert_combine(rows, plan, **k),
        "expert_combine_bwd": lambda **k: binding.gs_expert_combine_bwd(rows, plan, route.weights, x, **k).rows,
        "orthogonalize": lambda **k: binding.gs_orthogonalize(x, **k),
        "expert_route": lambda **k: binding.gs_expert_route(logits, K, **k).weights,
        "expert_route_bwd": lambda **k: binding.gs_expert_route_bwd(logits, route, route.weights, **k),
        "quantize": lambda **k: binding.gs_quantize(x, **k).scales,
        "dequantize": lambda **k: binding.gs_dequantize(q, **k),
        "expert_product": lambda **k: binding.gs_expert_product(q, qw, plan, gather=True, **k),
        "expert_weight_grad": lambda **k: binding.gs_expert_weight_grad(q, rows, plan, gather=True, **k),
    }


def test_another_device(monkeypatch):
    for name, call in calls().items():
        want = call()
        with monkeypatch.context() as m:
            m.setattr(torch.cuda, "current_device", lambda: 1)
            with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
                call()
        assert torch.equal(call(), want), name


def test_a_stream_of_the_same_device():
    for name, call in calls().items():
        want = call()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = call(stream=side)
        side.synchronize()
        assert torch.equal(got, want), name
