"""Host-side checks of the training operators (no GPU): the C ABI's refusals, the binding's, and the 64-bit forms the
GPU tests compare with (their gradients against differences, the update against a singular value decomposition)."""
import ctypes

import pytest
import torch

import train_util as tu
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


def test_layer_norm_refusals(lib):
    bad, space = binding.GS_ERR_INVALID_ARG, binding.GS_ERR_WORKSPACE

    def fwd(rows=4, dim=8, eps=1e-5, dt=0, wdt=0, x=FAKE, w=FAKE, y=FAKE, mean=FAKE, rstd=FAKE):
        return lib.gs_layer_norm_fwd(x, w, None, rows, dim, eps, dt, wdt, y, mean, rstd, None)
    for kw, word in ((dict(rows=-1), "rows"), (dict(rows=1 << 31), "rows"), (dict(dim=0), "dim"),
                     (dict(dim=1 << 31), "dim"), (dict(dt=3), "dtype"), (dict(dt=-1), "dtype"),
                     (dict(dt=1, wdt=2), "weight_dtype"), (dict(dt=0, wdt=1), "weight_dtype"),
                     (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(mean=None), "together"),
                     (dict(x=None), "NULL"), (dict(w=None), "NULL"), (dict(y=None), "NULL")):
        refused(lib, fwd(**kw), bad, word)
    assert fwd(rows=0, x=None, y=None) == binding.GS_OK  # nothing to do

    def bwd(rows=4, dim=8, dt=0, wdt=0, x=FAKE, gw=FAKE, ws=FAKE, wsb=1 << 20):
        return lib.gs_layer_norm_bwd(x, FAKE, FAKE, FAKE, FAKE, rows, dim, dt, wdt, FAKE, gw, None, ws, wsb, None)
    for kw, word in ((dict(rows=-1), "rows"), (dict(dim=0), "dim"), (dict(dt=7), "dtype"),
                     (dict(dt=2, wdt=1), "weight_dtype"), (dict(x=None), "NULL"), (dict(gw=None), "NULL")):
        refused(lib, bwd(**kw), bad, word)
    refused(lib, bwd(ws=None), space, "workspace")
    refused(lib, bwd(wsb=lib.gs_layer_norm_bwd_workspace_bytes(4, 8) - 1), space, "workspace")
    assert lib.gs_layer_norm_bwd_workspace_bytes(-1, 8) == 0
    assert lib.gs_layer_norm_bwd_workspace_bytes(1 << 20, 1 << 20) > 1 << 24


def test_expert_refusals(lib):
    bad, space = binding.GS_ERR_INVALID_ARG, binding.GS_ERR_WORKSPACE

    def plan(T=4, K=2, E=8, ids=FAKE, off=FAKE, ws=FAKE, wsb=1 << 30):
        return lib.gs_expert_plan(ids, T, K, E, off, FAKE, FAKE, ws, wsb, None)
    for kw, word in ((dict(T=-1), "tokens"), (dict(K=0), "choices"), (dict(T=1 << 20, K=1 << 11), "2^31"),
                     (dict(E=0), "experts"), (dict(E=4097), "experts"), (dict(ids=None), "NULL"),
                     (dict(off=None), "NULL")):
        refused(lib, plan(**kw), bad, word)
    big = lib.gs_expert_plan_workspace_bytes(1 << 20, 2, 8)
    assert big > 0
    refused(lib, plan(T=1 << 20, wsb=big - 1), space, "workspace")
    refused(lib, plan(T=1 << 20, ws=None), space, "workspace")
    assert lib.gs_expert_plan_workspace_bytes(1 << 20, 1 << 11, 8) == 0

    def dispatch(T=4, K=2, E=8, D=16, dt=0, x=FAKE):
        return lib.gs_expert_dispatch(x, FAKE, FAKE, T, K, E, D, dt, FAKE, None)

    def combine(T=4, K=2, E=8, D=16, dt=0, x=FAKE):
        return lib.gs_expert_combine(x, FAKE, None, T, K, D, dt, FAKE, None)

    def combine_bwd(T=4, K=2, E=8, D=16, dt=0, x=FAKE):
        return lib.gs_expert_combine_bwd(x, FAKE, FAKE, FAKE, FAKE, T, K, E, D, dt, FAKE, FAKE, None)
    for call in (dispatch, combine, combine_bwd):
        for kw, word in ((dict(T=-1), "tokens"), (dict(K=0), "choices"), (dict(D=0), "dim"), (dict(D=1 << 31), "dim"),
                         (dict(dt=3), "dtype"), (dict(x=None), "NULL")):
            refused(lib, call(**kw), bad, word)
        assert call(T=0, x=None) == binding.GS_OK
    refused(lib, dispatch(E=0), bad, "experts")


def test_orthogonalize_refusals(lib):
    bad, space = binding.GS_ERR_INVALID_ARG, binding.GS_ERR_WORKSPACE

    def ortho(B=1, m=8, n=8, steps=5, eps=1e-7, dt=0, u=FAKE, ws=FAKE, wsb=1 << 40):
        return lib.gs_orthogonalize(u, B, m, n, steps, 1.5, -0.5, 0.0, eps, dt, FAKE, ws, wsb, None)
    for kw, word in ((dict(m=0), "m, n"), (dict(n=65537), "m, n"), (dict(B=-1), "batch"), (dict(B=65536), "batch"),
                     (dict(B=65535, m=65536, n=65536), "2^40"), (dict(steps=-1), "steps"), (dict(steps=101), "steps"),
                     (dict(dt=3), "dtype"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
                     (dict(u=None), "NULL")):
        refused(lib, ortho(**kw), bad, word)
    need = lib.gs_orthogonalize_workspace_bytes(3, 300, 200)
    assert need > 0
    refused(lib, ortho(B=3, m=300, n=200, wsb=need - 1), space, "workspace")
    refused(lib, ortho(B=3, m=300, n=200, ws=None), space, "workspace")
    assert lib.gs_orthogonalize_workspace_bytes(3, 100, 60) == 0  # the chip's own memory holds a small matrix
    assert ortho(B=0, u=None) == binding.GS_OK
    for sizes in ((1, 0, 8), (1, 8, 65537), (0, 8, 8), (65535, 65536, 65536)):
        assert lib.gs_orthogonalize_workspace_bytes(*sizes) == 0
    assert lib.gs_orthogonalize_workspace_bytes(1, 65536, 65536) > 0  # no overflow at the largest matrix


def test_binding_refusals(lib):
    """Shapes, types and layouts are refused before the device is looked at, and the device before any launch."""
    f, h, i = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.float16), torch.zeros(4, 2, dtype=torch.int32)
    w = torch.zeros(8)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        binding.gs_layer_norm_fwd(f.double(), w.double())
    with pytest.raises(TypeError, match="weight must be"):
        binding.gs_layer_norm_fwd(f, w.half())
    with pytest.raises(TypeError, match="weight must be"):
        binding.gs_layer_norm_fwd(h, w.bfloat16())
    with pytest.raises(ValueError, match="contiguous"):
        binding.gs_layer_norm_fwd(torch.zeros(8, 4).T, w)
    with pytest.raises(ValueError, match="column"):
        binding.gs_layer_norm_fwd(torch.zeros(4, 0), torch.zeros(0))
    with pytest.raises(ValueError, match="GPU device"):
        binding.gs_layer_norm_fwd(f, w)
    plan = binding.ExpertPlan(torch.zeros(9, dtype=torch.int32), i, torch.zeros(8, dtype=torch.int32))
    with pytest.raises(TypeError, match="ids must be"):
        binding.gs_expert_plan(i.long(), 8)
    with pytest.raises(ValueError, match="GPU device"):
        binding.gs_expert_plan(i, 8)
    for call in (lambda: binding.gs_expert_dispatch(f, plan), lambda: binding.gs_expert_combine(f, plan),
                 lambda: binding.gs_expert_combine_bwd(f, plan, torch.zeros(4, 2), f)):
        with pytest.raises(ValueError, match="GPU device"):
            call()
    with pytest.raises(ValueError, match=r"\[m, n\]"):
        binding.gs_orthogonalize(torch.zeros(8))
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        binding.gs_orthogonalize(torch.zeros(8, 8, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU device"):
        binding.gs_orthogonalize(f)


def differences(f, x, h=1e-6):
    """Central differences of the number f(x) at every entry of the float64 tensor x."""
    g = torch.empty_like(x)
    for i in range(x.numel()):
        at = x.reshape(-1)[i].item()
        v = []
        for s in (h, -h):
            x.reshape(-1)[i] = at + s
            v.append(f(x).item())
        x.reshape(-1)[i] = at
        g.reshape(-1)[i] = (v[0] - v[1]) / (2 * h)
    return g


def test_layer_norm_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(1)
    x, gy = (torch.randn(3, 7, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = torch.randn(7, generator=g, dtype=torch.float64), torch.randn(7, generator=g, dtype=torch.float64)
    _, mean, rstd = tu.layer_norm(x, w, b, 1e-5)
    gx, gw, gb = tu.layer_norm_grad(x, w, mean, rstd, gy)
    # central differences of step 1e-6 are off by about 1e-12 of the third derivative and 1e-10 by cancellation
    for got, want in ((gx, differences(lambda v: (gy * tu.layer_norm(v, w, b, 1e-5)[0]).sum(), x)),
                      (gw, differences(lambda v: (gy * tu.layer_norm(x, v, b, 1e-5)[0]).sum(), w)),
                      (gb, differences(lambda v: (gy * tu.layer_norm(x, w, v, 1e-5)[0]).sum(), b))):
        torch.testing.assert_close(got, want, rtol=1e-7, atol=1e-8)


def test_expert_gradient_formulas_against_differences():
    g = torch.Generator().manual_seed(2)
    T, K, E, D = 5, 2, 3, 4
    ids = torch.randint(-1, E, (T, K), generator=g, dtype=torch.int32)
    _, rows, pairs = tu.expert_plan(ids, E)
    src, gy = torch.randn(T * K, D, generator=g, dtype=torch.float64), torch.randn(T, D, generator=g,
                                                                                  dtype=torch.float64)
    w = torch.rand(T, K, generator=g, dtype=torch.float64)
    gs, gw, _ = tu.expert_combine_grad(src, rows, w, gy)
    loss = lambda s, v: (gy * tu.expert_combine(s, rows, v)[0]).sum()  # noqa: E731
    torch.testing.assert_close(gs, differences(lambda v: loss(v, w), src), rtol=1e-7, atol=1e-8)
    torch.testing.assert_close(gw, differences(lambda v: loss(src, v), w), rtol=1e-7, atol=1e-8)
    # the dispatch's gradient is the combine without weights
    x, gr = torch.randn(T, D, generator=g, dtype=torch.float64), torch.randn(T * K, D, generator=g,
                                                                             dtype=torch.float64)
    gx = tu.expert_combine(gr, rows, None)[0]
    want = differences(lambda v: (gr * tu.expert_dispatch(v, pairs, K)).sum(), x)
    torch.testing.assert_close(gx, want, rtol=1e-7, atol=1e-8)


def test_orthogonalize_form_moves_singular_values_only():
    g = torch.Generator().manual_seed(3)
    for shape in ((6, 9), (9, 6), (7, 7)):
        u = torch.randn(shape, generator=g)
        got = tu.orthogonalize(u)
        left, s, right = torch.linalg.svd(u.double() / (u.double().norm() + 1e-7), full_matrices=False)
        a, b, c = tu.COEFFICIENTS
        for _ in range(5):
            s = a * s + b * s ** 3 + c * s ** 5
        torch.testing.assert_close(got, left @ torch.diag(s) @ right, rtol=1e-9, atol=1e-9)


def test_a_workspace_of_the_caller_is_looked_at():
    """A given workspace has to be bytes on the operands' device."""
    for bad in (torch.zeros(4, dtype=torch.float32), torch.zeros(4, dtype=torch.uint8), [1, 2]):
        with pytest.raises((TypeError, ValueError), match="workspace"):
            binding._given_room(bad, torch.device("cuda", 0))
