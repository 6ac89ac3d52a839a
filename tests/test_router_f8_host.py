"""Host-side checks of the router, of values held in 8 bits and of their products (no GPU): the C ABI's refusals, the
binding's, overlaps, and the 64-bit forms (the router's gradient against differences, the 8-bit grid against its
definition)."""
import ctypes

import pytest
import torch

import f8_util as fu
from test_training_host import differences
from tile_binned_gaussian_amd import binding

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails on the host first


@pytest.fixture(scope="module")
def lib():
    from tile_binned_gaussian_amd import build
    if build.stale():
        build.build()
    return binding.load_library()


def refused(lib, status, code, word):
    assert status == code
    assert word in lib.gs_last_error().decode()


BAD, SPACE = binding.GS_ERR_INVALID_ARG, binding.GS_ERR_WORKSPACE


def at(k):
    """Addresses far apart."""
    return ctypes.c_void_p(k << 40)


def test_route_refusals(lib):
    def fwd(T=4, E=8, K=2, dt=0, x=at(1), ids=at(2), loss=at(6), ws=at(9), wsb=1 << 30):
        return lib.gs_expert_route(x, None, T, E, K, 1, dt, ids, at(3), at(4), at(5), loss, at(7), ws, wsb, None)
    for kw, word in ((dict(T=-1), "tokens"), (dict(T=1 << 31), "tokens"), (dict(K=0), "choices"),
                     (dict(T=1 << 30, E=8, K=4), "2^31"), (dict(E=0), "experts"), (dict(E=4097), "experts"),
                     (dict(K=9), "choices"), (dict(dt=3), "dtype"), (dict(x=None), "NULL"), (dict(ids=None), "NULL"),
                     (dict(loss=None), "NULL"), (dict(T=0, loss=None), "NULL")):
        refused(lib, fwd(**kw), BAD, word)
    need = lib.gs_expert_route_workspace_bytes(100000, 8)
    assert need > 0
    refused(lib, fwd(T=100000, wsb=need - 1), SPACE, "workspace")
    refused(lib, fwd(T=100000, ws=None), SPACE, "workspace")
    assert lib.gs_expert_route_workspace_bytes(16, 8) == 0
    assert lib.gs_expert_route_workspace_bytes(16, 0) == 0 and lib.gs_expert_route_workspace_bytes(-1, 8) == 0

    def bwd(T=4, E=8, K=2, dt=0, x=at(1), kept=at(5), out=at(8)):
        return lib.gs_expert_route_bwd(x, at(2), at(3), at(4), kept, None, None, T, E, K, 1, dt, out, None)
    for kw, word in ((dict(T=-1), "tokens"), (dict(K=9), "choices"), (dict(E=4097, K=1), "experts"),
                     (dict(dt=-1), "dtype"), (dict(x=None), "NULL"), (dict(kept=None), "NULL"),
                     (dict(out=None), "NULL")):
        refused(lib, bwd(**kw), BAD, word)
    assert bwd(T=0, x=None) == binding.GS_OK


def test_held_refusals(lib):
    def q(B=1, R=4, D=8, t=0, dt=0, x=at(1), v=at(2), s=at(3)):
        return lib.gs_quantize(x, B, R, D, t, dt, v, s, None)
    for kw, word in ((dict(R=-1), "rows"), (dict(R=1 << 31), "rows"), (dict(D=0), "dim"), (dict(D=1 << 31), "dim"),
                     (dict(B=-1), "batch"), (dict(B=1 << 16, R=1 << 16), "batch"), (dict(dt=3), "dtype"),
                     (dict(B=1 << 16, D=1 << 16, R=1, t=1), "transpose"), (dict(x=None), "NULL"),
                     (dict(v=None), "NULL"), (dict(s=None), "NULL"), (dict(v=ctypes.c_void_p(0x1008)), "16")):
        refused(lib, q(**kw), BAD, word)
    assert q(R=0, x=None) == binding.GS_OK and q(B=0, x=None) == binding.GS_OK

    def d(R=4, D=8, dt=0, x=at(1), v=at(2), s=at(3)):
        return lib.gs_dequantize(v, s, R, D, dt, x, None)
    for kw, word in ((dict(R=-1), "rows"), (dict(D=0), "dim"), (dict(dt=9), "dtype"), (dict(x=None), "NULL"),
                     (dict(v=ctypes.c_void_p(0x1001)), "16")):
        refused(lib, d(**kw), BAD, word)
    assert d(R=0, x=None) == binding.GS_OK


def test_product_refusals(lib):
    def product(R=8, X=4, K=2, E=3, D=16, N=8, dt=1, x=at(1), w=at(3), off=at(5), pairs=at(6), out=at(7)):
        return lib.gs_expert_product(x, at(2), w, at(4), off, pairs, R, X, K, E, D, N, 0, dt, out, None)

    def grad(R=8, X=4, K=2, E=3, D=16, N=8, dt=1, x=at(1), w=at(3), off=at(5), pairs=at(6), out=at(7), ws=at(8),
             wsb=1 << 40):
        return lib.gs_expert_weight_grad(x, at(2), w, off, pairs, R, X, K, E, D, N, dt, out, ws, wsb, None)
    for call in (product, grad):
        for kw, word in ((dict(R=-1), "rows"), (dict(R=1 << 31), "rows"), (dict(X=-1), "rows"), (dict(E=0), "experts"),
                         (dict(E=4097), "experts"), (dict(off=None), "one expert"), (dict(D=0), "dim"),
                         (dict(N=0), "cols"), (dict(N=1 << 31), "cols"), (dict(dt=3), "dtype"), (dict(K=0), "choices"),
                         (dict(X=5), "go with"), (dict(pairs=None), "go with"), (dict(x=None), "NULL"),
                         (dict(w=None), "NULL"), (dict(out=None), "NULL"),
                         (dict(x=ctypes.c_void_p((1 << 40) + 8)), "16")):
            refused(lib, call(**kw), BAD, word)
    refused(lib, product(w=ctypes.c_void_p((3 << 40) + 4)), BAD, "16")
    assert product(R=0, X=0, x=None) == binding.GS_OK
    need = lib.gs_expert_weight_grad_workspace_bytes(400000, 8, 128, 256)
    assert need > 0
    big = dict(R=400000, X=200000, E=8, D=128, N=256)
    refused(lib, grad(**big, wsb=need - 1), SPACE, "workspace")
    refused(lib, grad(**big, ws=None), SPACE, "workspace")
    for sizes in ((-1, 8, 128, 256), (100, 0, 128, 256), (100, 8, 0, 256), (100, 8, 128, 1 << 31),
                  (400, 64, 4096, 4096)):
        assert lib.gs_expert_weight_grad_workspace_bytes(*sizes) == 0


R, D, N, T, K, E = 8, 200, 6, 4, 2, 3
BLOCKS = 2
ARRAYS = {
    "gs_expert_route": [("logits", 20000 * E * 4, 0), ("mask", 20000, 0), ("ids", 20000 * K * 4, 1),
                        ("weights", 20000 * K * 4, 1), ("counts", E * 4, 1), ("shares", E * 4, 1), ("loss", 4, 1),
                        ("kept", 4, 1), ("workspace", None, 1)],
    "gs_expert_route_bwd": [("logits", T * E * 4, 0), ("ids", T * K * 4, 0), ("weights", T * K * 4, 0),
                            ("counts", E * 4, 0), ("kept", 4, 0), ("grad_weights", T * K * 4, 0), ("grad_loss", 4, 0),
                            ("grad_logits", T * E * 4, 1)],
    "gs_quantize": [("x", R * D * 4, 0), ("values", R * BLOCKS * 128, 1), ("scales", R * BLOCKS, 1)],
    "gs_dequantize": [("values", R * BLOCKS * 128, 0), ("scales", R * BLOCKS, 0), ("x", R * D * 4, 1)],
    "gs_expert_product": [("x", T * BLOCKS * 128, 0), ("x_scales", T * BLOCKS, 0), ("weight", E * N * BLOCKS * 128, 0),
                          ("weight_scales", E * N * BLOCKS, 0), ("offsets", (E + 1) * 4, 0), ("pairs", R * 4, 0),
                          ("out", R * N * 4, 1)],
    "gs_expert_weight_grad": [("x", 5000 * BLOCKS * 128, 0), ("x_scales", 5000 * BLOCKS, 0),
                              ("grad", 10000 * N * 4, 0), ("offsets", (E + 1) * 4, 0), ("pairs", 10000 * 4, 0),
                              ("out", E * D * N * 4, 1), ("workspace", None, 1)],
}


def room(lib, name):
    return {"gs_expert_route": lambda: lib.gs_expert_route_workspace_bytes(20000, E),
            "gs_expert_weight_grad": lambda: lib.gs_expert_weight_grad_workspace_bytes(10000, E, D, N)}.get(
                name, lambda: 0)()


def call(lib, name, where):
    p = {k: ctypes.c_void_p(v) for k, v in where.items()}
    a = [p[k] for k, _, _ in ARRAYS[name]]
    ws = room(lib, name)
    return {
        "gs_expert_route": lambda: lib.gs_expert_route(*a[:2], 20000, E, K, 1, 0, *a[2:], ws, None),
        "gs_expert_route_bwd": lambda: lib.gs_expert_route_bwd(*a[:7], T, E, K, 1, 0, a[7], None),
        "gs_quantize": lambda: lib.gs_quantize(a[0], 1, R, D, 0, 0, *a[1:], None),
        "gs_dequantize": lambda: lib.gs_dequantize(*a[:2], R, D, 0, a[2], None),
        "gs_expert_product": lambda: lib.gs_expert_product(*a[:6], R, T, K, E, D, N, 0, 0, a[6], None),
        "gs_expert_weight_grad": lambda: lib.gs_expert_weight_grad(*a[:5], 10000, 5000, K, E, D, N, 0, *a[5:], ws, None),
    }[name]()


def pairs():
    for name, arrays in ARRAYS.items():
        for i, (a, _, wa) in enumerate(arrays):
            for b, _, wb in arrays[i + 1:]:
                if wa or wb:
                    yield pytest.param(name, a, b, id=f"{name}-{a}-{b}")


@pytest.mark.parametrize("name,a,b", pairs())
def test_overlaps_are_refused(lib, name, a, b):
    """One byte in common, and the same address (values lie at multiples of 16 bytes)."""
    size = {k: v if v is not None else room(lib, name) for k, v, _ in ARRAYS[name]}
    assert all(v > 0 for v in size.values())
    apart = {k: (i + 1) << 40 for i, k in enumerate(size)}
    for to in ((apart[a] + size[a] - 1) // 16 * 16, apart[a]):
        assert call(lib, name, {**apart, b: to}) == BAD
        message = lib.gs_last_error().decode()
        assert name in message and "overlaps" in message and a in message and b in message


def test_binding_refusals(lib):
    """Shapes, types and layouts are refused before the device is looked at, and the device before any launch."""
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="choices must be"):
        binding.gs_expert_route(x, 9)
    with pytest.raises(ValueError, match=r"\[tokens, experts\]"):
        binding.gs_expert_route(torch.zeros(4), 1)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        binding.gs_expert_route(x.double(), 2)
    with pytest.raises(ValueError, match="GPU device"):
        binding.gs_expert_route(x, 2)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        binding.gs_quantize(x.int())
    with pytest.raises(ValueError, match="dim"):
        binding.gs_quantize(torch.zeros(8), transpose=True)
    with pytest.raises(ValueError, match="dim"):
        binding.gs_quantize(torch.zeros(4, 0))
    with pytest.raises(ValueError, match="contiguous"):
        binding.gs_quantize(torch.zeros(8, 4).T)
    with pytest.raises(ValueError, match="GPU device"):
        binding.gs_quantize(x)
    with pytest.raises(TypeError, match="Quantized"):
        binding.gs_dequantize(x)
    held = binding.Quantized(torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.zeros(4, 1, dtype=torch.uint8), 8)
    for bad, word in ((binding.Quantized(held.values, held.scales, 129), "shape"),
                      (binding.Quantized(held.values, held.scales, 0), "column"),
                      (binding.Quantized(held.values, torch.zeros(4, 2, dtype=torch.uint8), 8), "shape"),
                      (binding.Quantized(held.values.view(torch.uint8), held.scales, 8), "float8"),
                      (held, "GPU device")):
        for f in (lambda q: binding.gs_dequantize(q), lambda q: binding.gs_expert_product(q, held),
                  lambda q: binding.gs_expert_weight_grad(q, x)):
            with pytest.raises((TypeError, ValueError), match=word):
                f(bad)


def test_router_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(1)
    T, E, K = 6, 5, 2
    x, gw = torch.randn(T, E, generator=g, dtype=torch.float64), torch.randn(T, K, generator=g, dtype=torch.float64)
    mask = torch.tensor([True, True, False, True, True, True])
    for renormalize in (True, False):
        ids, w, counts, _, _, kept = fu.route(x, K, mask, renormalize)
        got, _ = fu.route_grad(x, ids, w, counts, kept, gw, 0.7, renormalize)

        def value(v):
            r = fu.route(v, K, mask, renormalize, ids=ids)
            return (gw * r[1]).sum() + 0.7 * r[4]
        torch.testing.assert_close(got, differences(value, x), rtol=1e-7, atol=1e-8)
        wide = x.clone().requires_grad_()
        value(wide).backward()
        torch.testing.assert_close(got, wide.grad, rtol=1e-12, atol=1e-14)


def test_a_balanced_router_has_loss_one():
    """Every expert chosen as often, and of the same mean probability."""
    x = torch.eye(6, dtype=torch.float64) * 3
    _, _, counts, shares, loss, _ = fu.route(x, 1)
    assert counts.tolist() == [1] * 6 and abs(loss.item() - 1) < 1e-12 and (shares - 1 / 6).abs().max() < 1e-12


def test_held_values_are_the_nearest_of_the_grid():
    """Every e4m3 number by its bits, and each value's nearest among them."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()
    grid = codes[codes.isfinite()].unique()
    assert grid.max() == 448
    x = torch.randn(20, 300, generator=torch.Generator().manual_seed(2)) * torch.exp(
        3 * torch.randn(300, generator=torch.Generator().manual_seed(3)))
    q, scales = fu.quantize(x)
    v = torch.nn.functional.pad(x.double(), (0, 84)).unflatten(-1, (3, 128))
    scaled = v / fu.power(scales.double() - 127)[..., None]
    most = scaled.abs().amax(dim=-1)
    assert (most <= 448).all() and (most > 224).all()
    nearest = (scaled[..., None] - grid).abs().amin(dim=-1)
    assert torch.equal((scaled - q.unflatten(-1, (3, 128))).abs(), nearest)
