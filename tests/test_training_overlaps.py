"""Outputs of the training operators that overlap an input or each other are refused on the host (no GPU)."""
import ctypes

import pytest

from tile_binned_gaussian_amd import binding

R, D, T, K, E = 6, 16, 5, 2, 4  # sizes of every call here
F = 4  # bytes of an element

# each operator's arguments that are arrays: name, bytes, whether it is written
ARRAYS = {
    "gs_layer_norm_fwd": [("x", R * D * F, 0), ("weight", D * F, 0), ("bias", D * F, 0), ("y", R * D * F, 1),
                          ("mean", R * F, 1), ("rstd", R * F, 1)],
    "gs_layer_norm_bwd": [("x", R * D * F, 0), ("weight", D * F, 0), ("mean", R * F, 0), ("rstd", R * F, 0),
                          ("grad_y", R * D * F, 0), ("grad_x", R * D * F, 1), ("grad_weight", D * F, 1),
                          ("grad_bias", D * F, 1), ("workspace", None, 1)],
    "gs_expert_plan": [("ids", 9000 * K * F, 0), ("offsets", (E + 1) * F, 1), ("rows", 9000 * K * F, 1),
                       ("pairs", 9000 * K * F, 1), ("workspace", None, 1)],
    "gs_expert_dispatch": [("x", T * D * F, 0), ("offsets", (E + 1) * F, 0), ("rows", T * K * F, 0),
                           ("sent", T * K * D * F, 1)],
    "gs_expert_combine": [("source", T * K * D * F, 0), ("rows", T * K * F, 0), ("weights", T * K * F, 0),
                          ("y", T * D * F, 1)],
    "gs_expert_combine_bwd": [("source", T * K * D * F, 0), ("offsets", (E + 1) * F, 0), ("rows", T * K * F, 0),
                              ("weights", T * K * F, 0), ("grad_y", T * D * F, 0), ("grad_source", T * K * D * F, 1),
                              ("grad_weights", T * K * F, 1)],
    "gs_orthogonalize": [("update", 2 * 300 * 200 * F, 0), ("out", 2 * 300 * 200 * F, 1), ("workspace", None, 1)],
}


@pytest.fixture(scope="module")
def lib():
    from tile_binned_gaussian_amd import build
    if build.stale():
        build.build()
    return binding.load_library()


def room(lib, name):
    return {"gs_layer_norm_bwd": lambda: lib.gs_layer_norm_bwd_workspace_bytes(R, D),
            "gs_expert_plan": lambda: lib.gs_expert_plan_workspace_bytes(9000, K, E),
            "gs_orthogonalize": lambda: lib.gs_orthogonalize_workspace_bytes(2, 300, 200)}.get(name, lambda: 0)()


def call(lib, name, at):
    """The operator on arrays at these addresses, which are never dereferenced: without a GPU no launch succeeds."""
    p = {k: ctypes.c_void_p(v) for k, v in at.items()}
    ws = room(lib, name)
    return {
        "gs_layer_norm_fwd": lambda: lib.gs_layer_norm_fwd(p["x"], p["weight"], p["bias"], R, D, 1e-5, 0, 0, p["y"],
                                                           p["mean"], p["rstd"], None),
        "gs_layer_norm_bwd": lambda: lib.gs_layer_norm_bwd(p["x"], p["weight"], p["mean"], p["rstd"], p["grad_y"], R, D,
                                                           0, 0, p["grad_x"], p["grad_weight"], p["grad_bias"],
                                                           p["workspace"], ws, None),
        "gs_expert_plan": lambda: lib.gs_expert_plan(p["ids"], 9000, K, E, p["offsets"], p["rows"], p["pairs"],
                                                     p["workspace"], ws, None),
        "gs_expert_dispatch": lambda: lib.gs_expert_dispatch(p["x"], p["offsets"], p["rows"], T, K, E, D, 0, p["sent"],
                                                             None),
        "gs_expert_combine": lambda: lib.gs_expert_combine(p["source"], p["rows"], p["weights"], T, K, D, 0, p["y"],
                                                           None),
        "gs_expert_combine_bwd": lambda: lib.gs_expert_combine_bwd(p["source"], p["offsets"], p["rows"], p["weights"],
                                                                   p["grad_y"], T, K, E, D, 0, p["grad_source"],
                                                                   p["grad_weights"], None),
        "gs_orthogonalize": lambda: lib.gs_orthogonalize(p["update"], 2, 300, 200, 5, 1.5, -0.5, 0.0, 1e-7, 0, p["out"],
                                                         p["workspace"], ws, None),
    }[name]()


def pairs():
    for name, arrays in ARRAYS.items():
        for i, (a, _, wa) in enumerate(arrays):
            for b, _, wb in arrays[i + 1:]:
                if wa or wb:
                    yield pytest.param(name, a, b, id=f"{name}-{a}-{b}")


@pytest.mark.parametrize("name,a,b", pairs())
def test_overlaps_are_refused(lib, name, a, b):
    """One byte in common, from either side, and the same address."""
    size = {k: v if v is not None else room(lib, name) for k, v, _ in ARRAYS[name]}
    apart = {k: (i + 1) << 40 for i, k in enumerate(size)}
    for at in (apart[a] + size[a] - 1, apart[a] - size[b] + 1, apart[a]):
        if name == "gs_orthogonalize" and (a, b) == ("update", "out") and at == apart[a]:
            continue  # in place
        assert call(lib, name, {**apart, b: at}) == binding.GS_ERR_INVALID_ARG
        message = lib.gs_last_error().decode()
        assert name in message and "overlaps" in message and a in message and b in message


@pytest.mark.parametrize("name", ARRAYS)
def test_neighbours_are_not_refused(recorder, name):
    """Arrays that touch, in either order, are launched."""
    from test_training_launches import recorded
    lines = recorded(recorder, f"""
import sys
sys.path.insert(0, "tests")
import test_training_overlaps as t
for order in (1, -1):
    at, place = {{}}, 1 << 40
    for k, v, _ in t.ARRAYS[{name!r}][::order]:
        at[k] = place
        place += v if v is not None else t.room(lib, {name!r})
    assert t.call(lib, {name!r}, at) == 0, lib.gs_last_error()
""")
    assert sum(line[0] == "launch" for line in lines) >= 2


from test_training_launches import recorder  # noqa: E402, F401  (the fixture)
