"""Thin ctypes binding of libgs_raster (C ABI in include/gs_raster.h), one Python function per entry point.

Argument marshalling only: every step runs in the HIP library. PyTorch supplies device memory (tensors on a ROCm
device) and the stream (torch's current stream unless one is passed). The library must be built
(``python -m tile_binned_gaussian_amd.build``); loading fails loudly otherwise, and there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
from dataclasses import dataclass

import torch  # loads the HIP runtime first, so the library binds to the same one

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgs_raster.so")

GS_OK, GS_ERR_INVALID_ARG, GS_ERR_OUT_OF_GRID, GS_ERR_WORKSPACE, GS_ERR_DEVICE = range(5)
_STATUS = {1: "GS_ERR_INVALID_ARG", 2: "GS_ERR_OUT_OF_GRID", 3: "GS_ERR_WORKSPACE", 4: "GS_ERR_DEVICE"}

EXPORTS = ("gs_last_error", "gs_isect_workspace_bytes", "gs_isect_tiles", "gs_sort_workspace_bytes",
           "gs_sort_keys", "gs_tile_ranges_workspace_bytes", "gs_tile_ranges", "gs_rasterize_workspace_bytes",
           "gs_rasterize_fwd", "gs_rasterize_fwd_hwexp", "gs_rasterize_fwd_traced", "gs_rasterize_bwd",
           "gs_project_fwd", "gs_bin_tiles", "gs_rasterize_fwd_bins", "gs_set_spin_limit", "gs_device_check",
           "gs_sort_keys_static", "gs_layer_norm_fwd", "gs_layer_norm_bwd_workspace_bytes", "gs_layer_norm_bwd",
           "gs_expert_plan_workspace_bytes", "gs_expert_plan", "gs_expert_dispatch", "gs_expert_combine",
           "gs_expert_combine_bwd", "gs_orthogonalize_workspace_bytes", "gs_orthogonalize",
           "gs_expert_route_workspace_bytes", "gs_expert_route", "gs_expert_route_bwd", "gs_quantize",
           "gs_dequantize", "gs_expert_product", "gs_expert_weight_grad_workspace_bytes",
           "gs_expert_weight_grad")

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}  # gs_dtype


class GsError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH):
    """Loads libgs_raster.so and declares every exported signature."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run `python -m tile_binned_gaussian_amd.build` (hipcc, gfx950)")
    lib = ctypes.CDLL(path)
    P, I64, I32, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.gs_last_error.argtypes, lib.gs_last_error.restype = [], ctypes.c_char_p
    lib.gs_isect_workspace_bytes.argtypes = [I64, I64, I64, I32, I32, I32]
    lib.gs_isect_workspace_bytes.restype = SZ
    lib.gs_isect_tiles.argtypes = [P, P, I32, P, I64, I64, I32, I32, I32, I32, P, P, P, P, P, I64, P, SZ, P]
    lib.gs_isect_tiles.restype = I32
    lib.gs_sort_workspace_bytes.argtypes, lib.gs_sort_workspace_bytes.restype = [I64, I32], SZ
    lib.gs_sort_keys.argtypes, lib.gs_sort_keys.restype = [P, P, I64, I32, P, SZ, P], I32
    lib.gs_tile_ranges_workspace_bytes.argtypes, lib.gs_tile_ranges_workspace_bytes.restype = [], SZ
    lib.gs_tile_ranges.argtypes = [P, I64, I64, I32, I32, P, I32, P, SZ, P]
    lib.gs_tile_ranges.restype = I32
    lib.gs_rasterize_workspace_bytes.argtypes = [I64, I32, I32]
    lib.gs_rasterize_workspace_bytes.restype = SZ
    lib.gs_rasterize_fwd.argtypes = [P, P, P, P, P, I64, I64, I32, I32, I32, I32, I32, I32, P, P, I64, P, F, F, F,
                                     P, P, P, P, P, P, SZ, P]
    lib.gs_rasterize_fwd.restype = I32
    lib.gs_rasterize_fwd_hwexp.argtypes = [P, P, P, P, P, I64, I64, I32, I32, I32, I32, I32, I32, P, P, I64, P, F, F,
                                           F, P, P, P, P, P, P]
    lib.gs_rasterize_fwd_hwexp.restype = I32
    lib.gs_rasterize_fwd_traced.argtypes = [P, P, P, P, P, I64, I64, I32, I32, I32, I32, I32, I32, P, P, I64, P, F,
                                            F, F, I32, I32, P, P, P, P, P, P, P, P, SZ, P]
    lib.gs_rasterize_fwd_traced.restype = I32
    lib.gs_bin_tiles.argtypes = [P, P, I32, P, I64, I64, I32, I32, I32, I32, P, P, P]
    lib.gs_bin_tiles.restype = I32
    lib.gs_rasterize_fwd_bins.argtypes = [P, P, P, P, P, I64, I64, I32, I32, I32, I32, I32, I32, P, P, I32, F, F, F,
                                          P, P, P, P, P, P]
    lib.gs_rasterize_fwd_bins.restype = I32
    lib.gs_rasterize_bwd.argtypes = [P, P, P, P, P, I64, I64, I32, I32, I32, I32, I32, I32, P, P, I64, P, F, F,
                                     P, P, P, P, P, P, P, P, P, P, P]
    lib.gs_rasterize_bwd.restype = I32
    lib.gs_project_fwd.argtypes = [P, P, P, P, I64, I64, I32, I32, F, F, F, F, I32, P, P, P, P, P, P]
    lib.gs_project_fwd.restype = I32
    lib.gs_sort_keys_static.argtypes, lib.gs_sort_keys_static.restype = [P, P, I64, I32, P], I32
    lib.gs_set_spin_limit.argtypes, lib.gs_set_spin_limit.restype = [ctypes.c_uint32], ctypes.c_uint32
    lib.gs_device_check.argtypes, lib.gs_device_check.restype = [P], I32
    lib.gs_layer_norm_fwd.argtypes = [P, P, P, I64, I64, F, I32, I32, P, P, P, P]
    lib.gs_layer_norm_fwd.restype = I32
    lib.gs_layer_norm_bwd_workspace_bytes.argtypes, lib.gs_layer_norm_bwd_workspace_bytes.restype = [I64, I64], SZ
    lib.gs_layer_norm_bwd.argtypes = [P, P, P, P, P, I64, I64, I32, I32, P, P, P, P, SZ, P]
    lib.gs_layer_norm_bwd.restype = I32
    lib.gs_expert_plan_workspace_bytes.argtypes, lib.gs_expert_plan_workspace_bytes.restype = [I64, I64, I32], SZ
    lib.gs_expert_plan.argtypes, lib.gs_expert_plan.restype = [P, I64, I64, I32, P, P, P, P, SZ, P], I32
    lib.gs_expert_dispatch.argtypes = [P, P, P, I64, I64, I32, I64, I32, P, P]
    lib.gs_expert_dispatch.restype = I32
    lib.gs_expert_combine.argtypes, lib.gs_expert_combine.restype = [P, P, P, I64, I64, I64, I32, P, P], I32
    lib.gs_expert_combine_bwd.argtypes = [P, P, P, P, P, I64, I64, I32, I64, I32, P, P, P]
    lib.gs_expert_combine_bwd.restype = I32
    lib.gs_orthogonalize_workspace_bytes.argtypes, lib.gs_orthogonalize_workspace_bytes.restype = [I64, I64, I64], SZ
    lib.gs_orthogonalize.argtypes = [P, I64, I64, I64, I32, F, F, F, F, I32, P, P, SZ, P]
    lib.gs_orthogonalize.restype = I32
    lib.gs_expert_route_workspace_bytes.argtypes, lib.gs_expert_route_workspace_bytes.restype = [I64, I32], SZ
    lib.gs_expert_route.argtypes = [P, P, I64, I32, I64, I32, I32, P, P, P, P, P, P, P, SZ, P]
    lib.gs_expert_route.restype = I32
    lib.gs_expert_route_bwd.argtypes = [P, P, P, P, P, P, P, I64, I32, I64, I32, I32, P, P]
    lib.gs_expert_route_bwd.restype = I32
    lib.gs_quantize.argtypes, lib.gs_quantize.restype = [P, I64, I64, I64, I32, I32, P, P, P], I32
    lib.gs_dequantize.argtypes, lib.gs_dequantize.restype = [P, P, I64, I64, I32, P, P], I32
    lib.gs_expert_product.argtypes = [P, P, P, P, P, P, I64, I64, I64, I32, I64, I64, I32, I32, P, P]
    lib.gs_expert_product.restype = I32
    lib.gs_expert_weight_grad_workspace_bytes.argtypes = [I64, I32, I64, I64]
    lib.gs_expert_weight_grad_workspace_bytes.restype = SZ
    lib.gs_expert_weight_grad.argtypes = [P, P, P, P, P, I64, I64, I64, I32, I64, I64, I32, P, P, SZ, P]
    lib.gs_expert_weight_grad.restype = I32
    _lib = lib
    return lib


def _check(status: int):
    if status != GS_OK:
        raise GsError(status, _lib.gs_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_scoped(fn):
    """Runs fn with its `stream` argument (when one is given) as torch's current stream, so that every buffer the
    call allocates - workspaces, outputs, a grown workspace and the copy into it - belongs to the stream its
    kernels run on: torch's caching allocator then never hands such a buffer to another stream while work queued
    on this one may still use it, and the copy is ordered after the work that produced its source."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        stream = args[at] if len(args) > at else kwargs.get("stream")
        if stream is None:
            return fn(*args, **kwargs)
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    return wrapper


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _req_layout(t, name, dtype, shape=None):
    """Type, dtype, shape and contiguity of one argument (no device check)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _req(t, name, dtype, device=None, shape=None):
    _req_layout(t, name, dtype, shape)
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _workspace(nbytes, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


@dataclass
class Intersections:
    tiles_per_gauss: torch.Tensor  # [C, N] int32
    gauss_offsets: torch.Tensor  # [C*N] int32
    isect_ids: torch.Tensor  # [n] int64 (the u64 key bits)
    flatten_ids: torch.Tensor  # [n] int32
    n_isects: int


@_stream_scoped
def gs_isect_tiles(means2d, radii, depths, tile_size, tile_width, tile_height, sort=True, stream=None,
                   workspace=None) -> Intersections:
    """Both phases of gs_isect_tiles: count (synchronises once for the size), then emit (and sort)."""
    lib = load_library()
    dev = means2d.device
    _req(means2d, "means2d", torch.float32, dev)
    if means2d.dim() != 3 or means2d.shape[2] != 2:
        raise ValueError("means2d must be [C, N, 2]")
    C, N = means2d.shape[0], means2d.shape[1]
    _req(radii, "radii", torch.float32, dev)
    if tuple(radii.shape) == (C, N):
        rpg = 1
    elif tuple(radii.shape) == (C, N, 2):
        rpg = 2
    else:
        raise ValueError(f"radii must be [C, N] or [C, N, 2] (got {tuple(radii.shape)})")
    _req(depths, "depths", torch.float32, dev, (C, N))
    s = _stream(stream)
    tiles_per = torch.empty((C, N), dtype=torch.int32, device=dev)
    goff = torch.empty(C * N, dtype=torch.int32, device=dev)
    n_out = ctypes.c_int64(0)
    ws = workspace if workspace is not None else _workspace(
        lib.gs_isect_workspace_bytes(C, N, 0, tile_width, tile_height, int(bool(sort))), dev)
    _check(lib.gs_isect_tiles(_ptr(means2d), _ptr(radii), rpg, _ptr(depths), C, N, tile_size, tile_width,
                              tile_height, int(bool(sort)), _ptr(tiles_per), _ptr(goff), ctypes.byref(n_out), None,
                              None, 0, _ptr(ws), ws.numel(), s))
    n = int(n_out.value)
    keys = torch.empty(n, dtype=torch.int64, device=dev)
    ids = torch.empty(n, dtype=torch.int32, device=dev)
    if n == 0:
        return Intersections(tiles_per, goff, keys, ids, n)
    need = lib.gs_isect_workspace_bytes(C, N, n, tile_width, tile_height, int(bool(sort)))
    if ws.numel() < need:
        # phase 1 left the depth order at the start of the workspace; phase 2 reads it there
        prefix = lib.gs_isect_workspace_bytes(C, N, 0, tile_width, tile_height, int(bool(sort)))
        grown = _workspace(need, dev)
        grown[:prefix].copy_(ws[:prefix])
        ws = grown
    _check(lib.gs_isect_tiles(_ptr(means2d), _ptr(radii), rpg, _ptr(depths), C, N, tile_size, tile_width,
                              tile_height, int(bool(sort)), None, _ptr(goff), None, _ptr(keys), _ptr(ids), n,
                              _ptr(ws), ws.numel(), s))
    return Intersections(tiles_per, goff, keys, ids, n)


@_stream_scoped
def gs_sort_keys(keys, flatten_ids, end_bit=64, stream=None, workspace=None):
    """Stable in-place sort of (keys, flatten_ids) by bits [0, end_bit) of the keys."""
    lib = load_library()
    _req(keys, "keys", torch.int64)
    _req(flatten_ids, "flatten_ids", torch.int32, keys.device, (keys.numel(),))
    n = keys.numel()
    ws = workspace if workspace is not None else _workspace(lib.gs_sort_workspace_bytes(n, end_bit), keys.device)
    _check(lib.gs_sort_keys(_ptr(keys), _ptr(flatten_ids), n, end_bit, _ptr(ws), ws.numel(), _stream(stream)))
    return keys, flatten_ids


def gs_sort_keys_static(keys, flatten_ids, end_bit=64, stream=None):
    """gs_sort_keys without a workspace (the library's static scratch; at most 2^22 pairs; allocates nothing).
    Calls that overlap on one GPU race."""
    lib = load_library()
    _req(keys, "keys", torch.int64)
    _req(flatten_ids, "flatten_ids", torch.int32, keys.device, (keys.numel(),))
    _check(lib.gs_sort_keys_static(_ptr(keys), _ptr(flatten_ids), keys.numel(), end_bit, _stream(stream)))
    return keys, flatten_ids


def gs_set_spin_limit(limit: int) -> int:
    """Look-back rounds a sort partition may wait before it gives up (passes launched afterwards); returns the
    previous limit."""
    return int(load_library().gs_set_spin_limit(int(limit)))


def gs_device_check(stream=None):
    """Synchronises the stream, then raises GsError (GS_ERR_DEVICE) if a sort's bounded wait gave up on this GPU
    since the last check (the device error word is cleared either way)."""
    _check(load_library().gs_device_check(_stream(stream)))


@_stream_scoped
def gs_tile_ranges(sorted_keys, C, tile_width, tile_height, validate=False, out=None, stream=None,
                   workspace=None):
    """Per-tile offsets [C, th, tw] int32 of sorted keys (boundary detection)."""
    lib = load_library()
    _req(sorted_keys, "sorted_keys", torch.int64)
    dev = sorted_keys.device
    if out is None:
        out = torch.empty((C, tile_height, tile_width), dtype=torch.int32, device=dev)
    _req(out, "isect_offsets", torch.int32, dev, (C, tile_height, tile_width))
    ws = workspace if workspace is not None else _workspace(lib.gs_tile_ranges_workspace_bytes(), dev)
    _check(lib.gs_tile_ranges(_ptr(sorted_keys), sorted_keys.numel(), C, tile_width, tile_height, _ptr(out),
                              int(bool(validate)), _ptr(ws), ws.numel(), _stream(stream)))
    return out


@dataclass
class Render:
    render_colors: torch.Tensor  # [C, H, W, K]
    render_alphas: torch.Tensor  # [C, H, W]
    render_T: torch.Tensor  # [C, H, W]
    last_ids: torch.Tensor  # [C, H, W] int32


def _raster_inputs(means2d, conics, colors, opacities, backgrounds, isect_offsets, flatten_ids, masks):
    dev = means2d.device
    _req(means2d, "means2d", torch.float32, dev)
    C, N = means2d.shape[0], means2d.shape[1]
    _req(conics, "conics", torch.float32, dev, (C, N, 3))
    _req(colors, "colors", torch.float32, dev)
    if colors.dim() != 3 or tuple(colors.shape[:2]) != (C, N):
        raise ValueError("colors must be [C, N, K]")
    _req(opacities, "opacities", torch.float32, dev, (C, N))
    if backgrounds is not None:
        _req(backgrounds, "backgrounds", torch.float32, dev, (C, colors.shape[2]))
    _req(isect_offsets, "isect_offsets", torch.int32, dev)
    if isect_offsets.dim() != 3 or isect_offsets.shape[0] != C:
        raise ValueError("isect_offsets must be [C, th, tw]")
    _req(flatten_ids, "flatten_ids", torch.int32, dev)
    if masks is not None:
        _req(masks, "masks", torch.int32, dev, tuple(isect_offsets.shape))
    return dev, C, N, colors.shape[2], isect_offsets.shape[1], isect_offsets.shape[2]


def _render_out(C, height, width, K, dev):
    return Render(torch.empty((C, height, width, K), dtype=torch.float32, device=dev),
                  torch.empty((C, height, width), dtype=torch.float32, device=dev),
                  torch.empty((C, height, width), dtype=torch.float32, device=dev),
                  torch.empty((C, height, width), dtype=torch.int32, device=dev))


def _check_render_out(out, C, height, width, K, dev):
    """A caller-supplied output set must match the image batch (the kernels write every pixel of it): every
    field's layout is checked first, then its device."""
    fields = [(out.render_colors, "render_colors", torch.float32, (C, height, width, K)),
              (out.render_alphas, "render_alphas", torch.float32, (C, height, width)),
              (out.render_T, "render_T", torch.float32, (C, height, width)),
              (out.last_ids, "last_ids", torch.int32, (C, height, width))]
    fields = [f for i, f in enumerate(fields) if i < 2 or f[0] is not None]
    for t, name, dtype, shape in fields:
        _req_layout(t, name, dtype, shape)
    for t, name, dtype, shape in fields:
        _req(t, name, dtype, dev, shape)


def _n_isects(flatten_ids, n_isects):
    """The intersection count the kernels may index: flatten_ids' length, or a given count that fits in it."""
    n = flatten_ids.numel() if n_isects is None else int(n_isects)
    if n < 0 or n > flatten_ids.numel():
        raise ValueError(f"n_isects = {n} outside [0, flatten_ids.numel() = {flatten_ids.numel()}]")
    return n


def _check_eval_counts(eval_counts, dev):
    if eval_counts is not None:
        _req(eval_counts, "eval_counts", torch.int64, dev, (5,))


@_stream_scoped
def gs_rasterize_fwd(means2d, conics, colors, opacities, backgrounds, width, height, tile_size, isect_offsets,
                     flatten_ids, n_isects=None, alpha_cutoff=1.0 / 255.0, alpha_clamp=0.99,
                     transmittance_threshold=1e-4, out=None, stream=None, workspace=None, eval_counts=None,
                     masks=None) -> Render:
    """Front-to-back compositing of every tile; returns colours, 1 - T, T and the last composited index.

    eval_counts: optional int64 [5] device tensor that the launch adds to (evaluations by the definition, alpha >=
    cutoff, composited, evaluations executed, splats staged)."""
    lib = load_library()
    dev, C, N, K, th, tw = _raster_inputs(means2d, conics, colors, opacities, backgrounds, isect_offsets,
                                          flatten_ids, masks)
    n = _n_isects(flatten_ids, n_isects)
    _check_eval_counts(eval_counts, dev)
    if out is None:
        out = _render_out(C, height, width, K, dev)
    _check_render_out(out, C, height, width, K, dev)
    ws = workspace if workspace is not None else _workspace(lib.gs_rasterize_workspace_bytes(C, tw, th), dev)
    _check(lib.gs_rasterize_fwd(_ptr(means2d), _ptr(conics), _ptr(colors), _ptr(opacities), _ptr(backgrounds), C, N,
                                K, width, height, tile_size, tw, th, _ptr(isect_offsets), _ptr(flatten_ids), n,
                                _ptr(masks), float(alpha_cutoff), float(alpha_clamp), float(transmittance_threshold),
                                _ptr(out.render_colors), _ptr(out.render_alphas), _ptr(out.render_T),
                                _ptr(out.last_ids), _ptr(eval_counts), _ptr(ws), ws.numel(), _stream(stream)))
    return out


@_stream_scoped
def gs_rasterize_fwd_hwexp(means2d, conics, colors, opacities, backgrounds, width, height, tile_size, isect_offsets,
                           flatten_ids, n_isects=None, alpha_cutoff=1.0 / 255.0, alpha_clamp=0.99,
                           transmittance_threshold=1e-4, out=None, stream=None, eval_counts=None,
                           masks=None) -> Render:
    """gs_rasterize_fwd with the hardware exponential (faster; not bit-identical to the specified one)."""
    lib = load_library()
    dev, C, N, K, th, tw = _raster_inputs(means2d, conics, colors, opacities, backgrounds, isect_offsets,
                                          flatten_ids, masks)
    n = _n_isects(flatten_ids, n_isects)
    _check_eval_counts(eval_counts, dev)
    if out is None:
        out = _render_out(C, height, width, K, dev)
    _check_render_out(out, C, height, width, K, dev)
    _check(lib.gs_rasterize_fwd_hwexp(_ptr(means2d), _ptr(conics), _ptr(colors), _ptr(opacities), _ptr(backgrounds),
                                      C, N, K, width, height, tile_size, tw, th, _ptr(isect_offsets),
                                      _ptr(flatten_ids), n, _ptr(masks), float(alpha_cutoff), float(alpha_clamp),
                                      float(transmittance_threshold), _ptr(out.render_colors),
                                      _ptr(out.render_alphas), _ptr(out.render_T), _ptr(out.last_ids),
                                      _ptr(eval_counts), _stream(stream)))
    return out


@dataclass
class TracedRender(Render):
    trace_ids: torch.Tensor | None  # [C, H, W, max_splat_steps] int32 flat splat ids (past the count: unwritten)
    trace_counts: torch.Tensor | None  # [C, H, W] int32


@_stream_scoped
def gs_rasterize_fwd_traced(means2d, conics, colors, opacities, backgrounds, width, height, tile_size,
                            isect_offsets, flatten_ids, max_splat_steps, max_list_entries=-1, n_isects=None,
                            alpha_cutoff=1.0 / 255.0, alpha_clamp=0.99, transmittance_threshold=1e-4, trace=True,
                            out=None, stream=None, workspace=None, eval_counts=None, masks=None) -> TracedRender:
    """The traced forward: each tile's list cut to its first max_list_entries entries (negative: whole lists),
    each pixel stopped after max_splat_steps composited splats, and (trace=True) each pixel's composited flat splat
    ids recorded in order with their count. Entries of a trace row past its count are left unwritten."""
    lib = load_library()
    dev, C, N, K, th, tw = _raster_inputs(means2d, conics, colors, opacities, backgrounds, isect_offsets,
                                          flatten_ids, masks)
    S = int(max_splat_steps)
    if S < 0:
        raise ValueError("max_splat_steps must be >= 0")
    n = _n_isects(flatten_ids, n_isects)
    _check_eval_counts(eval_counts, dev)
    if out is None:
        r = _render_out(C, height, width, K, dev)
        out = TracedRender(r.render_colors, r.render_alphas, r.render_T, r.last_ids,
                           torch.empty((C, height, width, S), dtype=torch.int32, device=dev) if trace else None,
                           torch.empty((C, height, width), dtype=torch.int32, device=dev) if trace else None)
    _check_render_out(out, C, height, width, K, dev)
    if out.trace_ids is not None:
        _req(out.trace_ids, "trace_ids", torch.int32, dev, (C, height, width, S))
    if out.trace_counts is not None:
        _req(out.trace_counts, "trace_counts", torch.int32, dev, (C, height, width))
    ws = workspace if workspace is not None else _workspace(lib.gs_rasterize_workspace_bytes(C, tw, th), dev)
    _check(lib.gs_rasterize_fwd_traced(_ptr(means2d), _ptr(conics), _ptr(colors), _ptr(opacities), _ptr(backgrounds),
                                       C, N, K, width, height, tile_size, tw, th, _ptr(isect_offsets),
                                       _ptr(flatten_ids), n, _ptr(masks), float(alpha_cutoff), float(alpha_clamp),
                                       float(transmittance_threshold), int(max_list_entries), S,
                                       _ptr(out.render_colors), _ptr(out.render_alphas), _ptr(out.render_T),
                                       _ptr(out.last_ids), _ptr(out.trace_ids), _ptr(out.trace_counts),
                                       _ptr(eval_counts), _ptr(ws), ws.numel(), _stream(stream)))
    return out


@dataclass
class Bins:
    bin_ids: torch.Tensor  # [C, th, tw, capacity] int32, -1 in empty slots
    bin_counts: torch.Tensor  # [C, th, tw] int32 full counts (> capacity: the bin overflowed)


@_stream_scoped
def gs_bin_tiles(means2d, radii, depths, tile_size, tile_width, tile_height, capacity, out=None,
                 stream=None) -> Bins:
    """Fixed-capacity per-tile bins: each tile's splats in (depth, id) order, -1 after them, and full counts."""
    lib = load_library()
    dev = means2d.device
    _req(means2d, "means2d", torch.float32, dev)
    if means2d.dim() != 3 or means2d.shape[2] != 2:
        raise ValueError("means2d must be [C, N, 2]")
    C, N = means2d.shape[0], means2d.shape[1]
    _req(radii, "radii", torch.float32, dev)
    if tuple(radii.shape) == (C, N):
        rpg = 1
    elif tuple(radii.shape) == (C, N, 2):
        rpg = 2
    else:
        raise ValueError(f"radii must be [C, N] or [C, N, 2] (got {tuple(radii.shape)})")
    _req(depths, "depths", torch.float32, dev, (C, N))
    if out is None:
        out = Bins(torch.empty((C, tile_height, tile_width, int(capacity)), dtype=torch.int32, device=dev),
                   torch.empty((C, tile_height, tile_width), dtype=torch.int32, device=dev))
    _req(out.bin_ids, "bin_ids", torch.int32, dev, (C, tile_height, tile_width, int(capacity)))
    _req(out.bin_counts, "bin_counts", torch.int32, dev, (C, tile_height, tile_width))
    _check(lib.gs_bin_tiles(_ptr(means2d), _ptr(radii), rpg, _ptr(depths), C, N, tile_size, tile_width, tile_height,
                            int(capacity), _ptr(out.bin_ids), _ptr(out.bin_counts), _stream(stream)))
    return out


@_stream_scoped
def gs_rasterize_fwd_bins(means2d, conics, colors, opacities, backgrounds, width, height, tile_size, bin_ids,
                          bin_counts, alpha_cutoff=1.0 / 255.0, alpha_clamp=0.99, transmittance_threshold=1e-4,
                          out=None, stream=None, eval_counts=None) -> Render:
    """Front-to-back compositing over fixed-capacity bins; last ids are bin positions t * capacity + m."""
    lib = load_library()
    dev = means2d.device
    _req(bin_ids, "bin_ids", torch.int32, dev)
    if bin_ids.dim() != 4:
        raise ValueError("bin_ids must be [C, th, tw, capacity]")
    _, C, N, K, th, tw = _raster_inputs(means2d, conics, colors, opacities, backgrounds, bin_counts,
                                        bin_ids, None)
    if tuple(bin_ids.shape[:3]) != (C, th, tw):
        raise ValueError("bin_ids and bin_counts disagree on [C, th, tw]")
    _check_eval_counts(eval_counts, dev)
    if out is None:
        out = _render_out(C, height, width, K, dev)
    _check_render_out(out, C, height, width, K, dev)
    _check(lib.gs_rasterize_fwd_bins(_ptr(means2d), _ptr(conics), _ptr(colors), _ptr(opacities), _ptr(backgrounds),
                                     C, N, K, width, height, tile_size, tw, th, _ptr(bin_ids), _ptr(bin_counts),
                                     bin_ids.shape[3], float(alpha_cutoff), float(alpha_clamp),
                                     float(transmittance_threshold), _ptr(out.render_colors), _ptr(out.render_alphas),
                                     _ptr(out.render_T), _ptr(out.last_ids), _ptr(eval_counts), _stream(stream)))
    return out


@dataclass
class RasterGrad:
    means2d: torch.Tensor  # [C, N, 2]
    conics: torch.Tensor  # [C, N, 3]
    colors: torch.Tensor  # [C, N, K]
    opacities: torch.Tensor  # [C, N]
    backgrounds: torch.Tensor | None  # [C, K]
    means2d_abs: torch.Tensor | None  # [C, N, 2]


@_stream_scoped
def gs_rasterize_bwd(means2d, conics, colors, opacities, backgrounds, width, height, tile_size, isect_offsets,
                     flatten_ids, render_alphas, last_ids, grad_render_colors, grad_render_alphas, n_isects=None,
                     alpha_cutoff=1.0 / 255.0, alpha_clamp=0.99, grad_backgrounds=None, absgrad=False, out=None,
                     stream=None, masks=None) -> RasterGrad:
    """Gradients of sum(grad_render_colors * colours) + sum(grad_render_alphas * alphas) of gs_rasterize_fwd.

    grad_backgrounds: None -> computed when backgrounds is given; False -> not computed."""
    lib = load_library()
    dev = means2d.device
    _req(means2d, "means2d", torch.float32, dev)
    C, N = means2d.shape[0], means2d.shape[1]
    _req(conics, "conics", torch.float32, dev, (C, N, 3))
    _req(colors, "colors", torch.float32, dev)
    if colors.dim() != 3 or tuple(colors.shape[:2]) != (C, N):
        raise ValueError("colors must be [C, N, K]")
    K = colors.shape[2]
    _req(opacities, "opacities", torch.float32, dev, (C, N))
    if backgrounds is not None:
        _req(backgrounds, "backgrounds", torch.float32, dev, (C, K))
    _req(isect_offsets, "isect_offsets", torch.int32, dev)
    th, tw = isect_offsets.shape[1], isect_offsets.shape[2]
    _req(flatten_ids, "flatten_ids", torch.int32, dev)
    _req(render_alphas, "render_alphas", torch.float32, dev, (C, height, width))
    _req(last_ids, "last_ids", torch.int32, dev, (C, height, width))
    _req(grad_render_colors, "grad_render_colors", torch.float32, dev, (C, height, width, K))
    _req(grad_render_alphas, "grad_render_alphas", torch.float32, dev, (C, height, width))
    n = _n_isects(flatten_ids, n_isects)
    if isect_offsets.dim() != 3 or isect_offsets.shape[0] != C:
        raise ValueError("isect_offsets must be [C, th, tw]")
    want_bg = backgrounds is not None if grad_backgrounds is None else bool(grad_backgrounds)
    if out is None:
        e = lambda *shape: torch.empty(shape, dtype=torch.float32, device=dev)  # noqa: E731
        out = RasterGrad(e(C, N, 2), e(C, N, 3), e(C, N, K), e(C, N), e(C, K) if want_bg else None,
                         e(C, N, 2) if absgrad else None)
    _req(out.means2d, "grad_means2d", torch.float32, dev, (C, N, 2))
    _req(out.conics, "grad_conics", torch.float32, dev, (C, N, 3))
    _req(out.colors, "grad_colors", torch.float32, dev, (C, N, K))
    _req(out.opacities, "grad_opacities", torch.float32, dev, (C, N))
    if out.backgrounds is not None:
        _req(out.backgrounds, "grad_backgrounds", torch.float32, dev, (C, K))
    if out.means2d_abs is not None:
        _req(out.means2d_abs, "grad_means2d_abs", torch.float32, dev, (C, N, 2))
    if masks is not None:
        _req(masks, "masks", torch.int32, dev, (C, th, tw))
    _check(lib.gs_rasterize_bwd(_ptr(means2d), _ptr(conics), _ptr(colors), _ptr(opacities), _ptr(backgrounds), C, N,
                                K, width, height, tile_size, tw, th, _ptr(isect_offsets), _ptr(flatten_ids), n,
                                _ptr(masks), float(alpha_cutoff), float(alpha_clamp), _ptr(render_alphas),
                                _ptr(last_ids), _ptr(grad_render_colors), _ptr(grad_render_alphas), _ptr(out.means2d),
                                _ptr(out.conics), _ptr(out.colors), _ptr(out.opacities), _ptr(out.backgrounds),
                                _ptr(out.means2d_abs), _stream(stream)))
    return out


@dataclass
class Projection:
    radii: torch.Tensor  # [C, N, 2] int32
    means2d: torch.Tensor  # [C, N, 2]
    depths: torch.Tensor  # [C, N]
    conics: torch.Tensor  # [C, N, 3]
    compensations: torch.Tensor | None  # [C, N]


@_stream_scoped
def gs_project_fwd(means, covars, viewmats, Ks, width, height, eps2d=0.3, near_plane=0.01, far_plane=1e10,
                   radius_clip=0.0, compensation=False, orthographic=False, out=None, stream=None) -> Projection:
    """EWA projection of [N, 3] means and [N, 3, 3] covariances into C cameras."""
    lib = load_library()
    dev = means.device
    _req(means, "means", torch.float32, dev)
    if means.dim() != 2 or means.shape[1] != 3:
        raise ValueError("means must be [N, 3]")
    N = means.shape[0]
    _req(covars, "covars", torch.float32, dev, (N, 3, 3))
    _req(viewmats, "viewmats", torch.float32, dev)
    if viewmats.dim() != 3 or tuple(viewmats.shape[1:]) != (4, 4):
        raise ValueError("viewmats must be [C, 4, 4]")
    C = viewmats.shape[0]
    _req(Ks, "Ks", torch.float32, dev, (C, 3, 3))
    if out is None:
        out = Projection(torch.empty((C, N, 2), dtype=torch.int32, device=dev),
                         torch.empty((C, N, 2), dtype=torch.float32, device=dev),
                         torch.empty((C, N), dtype=torch.float32, device=dev),
                         torch.empty((C, N, 3), dtype=torch.float32, device=dev),
                         torch.empty((C, N), dtype=torch.float32, device=dev) if compensation else None)
    _check(lib.gs_project_fwd(_ptr(means), _ptr(covars), _ptr(viewmats), _ptr(Ks), C, N, int(width), int(height),
                              float(eps2d), float(near_plane), float(far_plane), float(radius_clip),
                              int(bool(orthographic)), _ptr(out.radii), _ptr(out.means2d), _ptr(out.depths),
                              _ptr(out.conics), _ptr(out.compensations), _stream(stream)))
    return out


# ----------------------------------------------------------------------------------------------------------------
# Training operators of a layer of experts


def _element(t, name):
    """The gs_dtype code of a tensor of one of the three element types."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16 (got {t.dtype})")
    return code


# These operators run on a handful of tokens too, where a call's cost is its host work: one look at an argument that is
# as it should be, and plain integers for ctypes. What is not as it should be goes to _req, which says why.


def _arg(t, name, dtype, device, shape):
    """The address of a tensor argument of this type, device and shape."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda
            and t.device == device):
        _req(t, name, dtype, device, shape)
    return t.data_ptr()


def _int32(v, name):
    """v as a C int; ctypes would cut it to 32 bits."""
    v = int(v)
    if not -(1 << 31) <= v < 1 << 31:
        raise ValueError(f"{name} must fit 32 bits (got {v})")
    return v


def _stream_int(stream, device):
    """The stream's handle. It has to be one of the tensors' device: a kernel on another one would read memory that is
    not its own, in no order with the work that fills it."""
    current = torch.cuda.current_device()  # a given stream's, where there is one
    if device.index != current:
        raise ValueError(f"the tensors are on {device}, the call's stream is on cuda:{current}: make theirs the "
                         "current device or pass one of its streams")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(current)
    return stream.cuda_stream


def _room(nbytes, device):
    """(workspace or None, its address, its size)."""
    if nbytes == 0:
        return None, None, 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), nbytes


def _given_room(workspace, device):
    _req(workspace, "workspace", torch.uint8, device)
    return workspace, workspace.data_ptr(), workspace.numel()


def _norm_inputs(x, weight):
    code, wcode = _element(x, "x"), _element(weight, "weight")
    if x.dim() < 1:
        raise ValueError("x must be [..., dim]")
    dim = x.shape[-1]
    if dim < 1:
        raise ValueError("x must have at least one column")
    if wcode not in (code, 0):
        raise TypeError(f"weight must be {x.dtype} or torch.float32 (got {weight.dtype})")
    dev = x.device
    return code, wcode, dev, x.numel() // dim, dim, _arg(x, "x", x.dtype, dev, x.shape), \
        _arg(weight, "weight", weight.dtype, dev, (dim,))


@dataclass
class LayerNorm:
    y: torch.Tensor  # x's shape and type
    mean: torch.Tensor | None  # [...] float32
    rstd: torch.Tensor | None  # [...] float32


@_stream_scoped
def gs_layer_norm_fwd(x, weight, bias=None, eps=1e-5, stats=True, out=None, stream=None) -> LayerNorm:
    """Layer norm over the last axis: y = (x - mean) * rstd * weight + bias with the rows' mean and rstd = 1 /
    sqrt(variance + eps) in float32 (stats=False: not returned).

    x [..., dim] of float32, bfloat16 or float16; weight and bias [dim] of x's type or float32."""
    lib = load_library()
    code, wcode, dev, rows, dim, px, pw = _norm_inputs(x, weight)
    pb = None if bias is None else _arg(bias, "bias", weight.dtype, dev, (dim,))
    shape = x.shape[:-1]
    if out is None:
        y, mean, rstd, pm, pr = torch.empty_like(x), None, None, None, None
        if stats:
            mean = torch.empty(shape, dtype=torch.float32, device=dev)
            rstd = torch.empty_like(mean)
            pm, pr = mean.data_ptr(), rstd.data_ptr()
        out, py = LayerNorm(y, mean, rstd), y.data_ptr()
    else:
        py, pm, pr = _arg(out.y, "y", x.dtype, dev, x.shape), None, None
        if (out.mean is None) != (out.rstd is None):
            raise ValueError("mean and rstd go together")
        if out.mean is not None:
            pm = _arg(out.mean, "mean", torch.float32, dev, shape)
            pr = _arg(out.rstd, "rstd", torch.float32, dev, shape)
    _check(lib.gs_layer_norm_fwd(px, pw, pb, rows, dim, eps, code, wcode, py, pm, pr, _stream_int(stream, dev)))
    return out


@dataclass
class LayerNormGrad:
    x: torch.Tensor  # x's shape and type
    weight: torch.Tensor  # [dim] of the weight's type
    bias: torch.Tensor | None  # [dim] of the weight's type


@_stream_scoped
def gs_layer_norm_bwd(x, weight, mean, rstd, grad_y, grad_bias=True, out=None, stream=None,
                      workspace=None) -> LayerNormGrad:
    """Gradients of sum(grad_y * y) of gs_layer_norm_fwd, from its inputs and statistics (grad_bias=False: the bias's
    is not computed)."""
    lib = load_library()
    code, wcode, dev, rows, dim, px, pw = _norm_inputs(x, weight)
    pm = _arg(mean, "mean", torch.float32, dev, x.shape[:-1])
    pr = _arg(rstd, "rstd", torch.float32, dev, x.shape[:-1])
    pg = _arg(grad_y, "grad_y", x.dtype, dev, x.shape)
    if out is None:
        out = LayerNormGrad(torch.empty_like(x), torch.empty_like(weight),
                            torch.empty_like(weight) if grad_bias else None)
        ox, ow, ob = out.x.data_ptr(), out.weight.data_ptr(), out.bias.data_ptr() if grad_bias else None
    else:
        ox = _arg(out.x, "grad_x", x.dtype, dev, x.shape)
        ow = _arg(out.weight, "grad_weight", weight.dtype, dev, (dim,))
        ob = None if out.bias is None else _arg(out.bias, "grad_bias", weight.dtype, dev, (dim,))
    ws, pws, room = _room(lib.gs_layer_norm_bwd_workspace_bytes(rows, dim), dev) if workspace is None \
        else _given_room(workspace, dev)
    _check(lib.gs_layer_norm_bwd(px, pw, pm, pr, pg, rows, dim, code, wcode, ox, ow, ob, pws, room,
                                 _stream_int(stream, dev)))
    return out


@dataclass
class ExpertPlan:
    offsets: torch.Tensor  # [experts + 1] int32: expert e has rows [offsets[e], offsets[e + 1])
    rows: torch.Tensor  # [tokens, choices] int32: each pair's row, -1 if dropped
    pairs: torch.Tensor  # [tokens * choices] int32: each row's pair, -1 past the kept ones


def _plan_inputs(plan, device):
    """(tokens, choices, experts, address of offsets, address of rows)."""
    rows, offsets = plan.rows, plan.offsets
    po, pr = _arg(offsets, "offsets", torch.int32, device, offsets.shape), _arg(rows, "rows", torch.int32, device,
                                                                                 rows.shape)
    if rows.dim() != 2 or rows.shape[1] < 1:
        raise ValueError("rows must be [tokens, choices]")
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must be [experts + 1]")
    return rows.shape[0], rows.shape[1], offsets.shape[0] - 1, po, pr


@_stream_scoped
def gs_expert_plan(ids, experts, out=None, stream=None, workspace=None) -> ExpertPlan:
    """The (token, choice) pairs of ids [tokens, choices] int32 in stable order of their expert; an id outside
    [0, experts) drops its pair."""
    lib = load_library()
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    pi = _arg(ids, "ids", torch.int32, ids.device, ids.shape)
    if ids.dim() != 2 or ids.shape[1] < 1:
        raise ValueError("ids must be [tokens, choices]")
    dev = ids.device
    (T, K), E = ids.shape, _int32(experts, "experts")
    if E < 1:
        raise ValueError("experts must be >= 1")
    if out is None:
        out = ExpertPlan(ids.new_empty(E + 1), torch.empty_like(ids), ids.new_empty(T * K))
        po, pr, pp = out.offsets.data_ptr(), out.rows.data_ptr(), out.pairs.data_ptr()
    else:
        po = _arg(out.offsets, "offsets", torch.int32, dev, (E + 1,))
        pr, pp = _arg(out.rows, "rows", torch.int32, dev, (T, K)), _arg(out.pairs, "pairs", torch.int32, dev, (T * K,))
    ws, pws, room = _room(lib.gs_expert_plan_workspace_bytes(T, K, E), dev) if workspace is None \
        else _given_room(workspace, dev)
    _check(lib.gs_expert_plan(pi, T, K, E, po, pr, pp, pws, room, _stream_int(stream, dev)))
    return out


@_stream_scoped
def gs_expert_dispatch(x, plan, out=None, stream=None):
    """Each token's row of x [tokens, dim] copied to its pairs' rows: [tokens * choices, dim], zeros in the rows past
    the kept ones. The gradient of x is gs_expert_combine(gradient of the result, plan)."""
    lib = load_library()
    code, dev = _element(x, "x"), x.device
    T, K, E, po, pr = _plan_inputs(plan, dev)
    if x.dim() != 2 or x.shape[0] != T or x.shape[1] < 1:
        raise ValueError(f"x must be [{T}, dim] (got {tuple(x.shape)})")
    px, D = _arg(x, "x", x.dtype, dev, x.shape), x.shape[1]
    if out is None:
        out = x.new_empty((T * K, D))
    else:
        _arg(out, "sent", x.dtype, dev, (T * K, D))
    _check(lib.gs_expert_dispatch(px, po, pr, T, K, E, D, code, out.data_ptr(), _stream_int(stream, dev)))
    return out


def _sorted_rows(t, name, T, K):
    if t.dim() != 2 or t.shape[0] != T * K or t.shape[1] < 1:
        raise ValueError(f"{name} must be [{T * K}, dim] (got {tuple(t.shape)})")
    return t.shape[1]


@_stream_scoped
def gs_expert_combine(source, plan, weights=None, out=None, stream=None):
    """Each token's sum of weights [tokens, choices] (float32; None: ones) times its kept pairs' rows of source
    [tokens * choices, dim]: [tokens, dim], summed in float32."""
    lib = load_library()
    code, dev = _element(source, "source"), source.device
    T, K, _, _, pr = _plan_inputs(plan, dev)
    D = _sorted_rows(source, "source", T, K)
    ps = _arg(source, "source", source.dtype, dev, source.shape)
    pw = None if weights is None else _arg(weights, "weights", torch.float32, dev, (T, K))
    if out is None:
        out = source.new_empty((T, D))
    else:
        _arg(out, "y", source.dtype, dev, (T, D))
    _check(lib.gs_expert_combine(ps, pr, pw, T, K, D, code, out.data_ptr(), _stream_int(stream, dev)))
    return out


@dataclass
class ExpertCombineGrad:
    rows: torch.Tensor  # [tokens * choices, dim], source's type
    weights: torch.Tensor  # [tokens, choices] float32


@_stream_scoped
def gs_expert_combine_bwd(source, plan, weights, grad_y, out=None, stream=None) -> ExpertCombineGrad:
    """Gradients of sum(grad_y * gs_expert_combine(source, plan, weights)) for source (zeros in the rows past the
    kept ones) and weights (0 for a dropped pair)."""
    lib = load_library()
    code, dev = _element(source, "source"), source.device
    T, K, E, po, pr = _plan_inputs(plan, dev)
    D = _sorted_rows(source, "source", T, K)
    ps = _arg(source, "source", source.dtype, dev, source.shape)
    pw = _arg(weights, "weights", torch.float32, dev, (T, K))
    pg = _arg(grad_y, "grad_y", source.dtype, dev, (T, D))
    if out is None:
        out = ExpertCombineGrad(torch.empty_like(source), torch.empty_like(weights))
    else:
        _arg(out.rows, "grad_rows", source.dtype, dev, (T * K, D))
        _arg(out.weights, "grad_weights", torch.float32, dev, (T, K))
    _check(lib.gs_expert_combine_bwd(ps, po, pr, pw, pg, T, K, E, D, code, out.rows.data_ptr(),
                                     out.weights.data_ptr(), _stream_int(stream, dev)))
    return out


@_stream_scoped
def gs_orthogonalize(update, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, out=None, stream=None,
                     workspace=None):
    """The orthogonalised update of each matrix of update [m, n] or [batch, m, n]: X = update / (|update| + eps), then
    `steps` times X = a X + (b A + c A A) X with A = X X^T and (a, b, c) = coefficients. out may be update."""
    lib = load_library()
    code, dev = _element(update, "update"), update.device
    if update.dim() not in (2, 3) or update.shape[-1] < 1 or update.shape[-2] < 1:
        raise ValueError(f"update must be [m, n] or [batch, m, n] (got {tuple(update.shape)})")
    pu = _arg(update, "update", update.dtype, dev, update.shape)
    m, n = update.shape[-2], update.shape[-1]
    B = update.shape[0] if update.dim() == 3 else 1
    (a, b, c), steps = coefficients, _int32(steps, "steps")
    if out is None:
        out = torch.empty_like(update)
    else:
        _arg(out, "out", update.dtype, dev, update.shape)
    ws, pws, room = _room(lib.gs_orthogonalize_workspace_bytes(B, m, n), dev) if workspace is None \
        else _given_room(workspace, dev)
    _check(lib.gs_orthogonalize(pu, B, m, n, steps, a, b, c, eps, code, out.data_ptr(), pws, room,
                                _stream_int(stream, dev)))
    return out


# ----------------------------------------------------------------------------------------------------------------
# The router of a layer of experts


@dataclass
class ExpertRoute:
    ids: torch.Tensor  # [tokens, choices] int32: the experts, best first; -1 where there is none
    weights: torch.Tensor  # [tokens, choices] float32
    counts: torch.Tensor  # [experts] int32: pairs of each expert
    shares: torch.Tensor  # [experts] float32: mean probability over the routed tokens
    loss: torch.Tensor  # [] float32: the balance loss
    kept: torch.Tensor  # [1] int32: tokens that were routed


def _logits(logits, choices):
    code = _element(logits, "logits")
    if logits.dim() != 2 or logits.shape[1] < 1:
        raise ValueError(f"logits must be [tokens, experts] (got {tuple(logits.shape)})")
    T, E = logits.shape
    if not 1 <= choices <= E:
        raise ValueError(f"choices must be in [1, experts = {E}] (got {choices})")
    return code, logits.device, T, _int32(E, "experts"), _arg(logits, "logits", logits.dtype, logits.device, (T, E))


@_stream_scoped
def gs_expert_route(logits, choices, mask=None, renormalize=True, out=None, stream=None, workspace=None) -> ExpertRoute:
    """Each token's `choices` best experts of logits [tokens, experts] with their weights (softmax over the chosen
    logits; renormalize=False: over all), the experts' counts and mean probabilities and the balance loss, experts *
    sum(counts / sum(counts) * shares). mask [tokens] bool: tokens to route; a logit of -inf is never chosen."""
    lib = load_library()
    K = int(choices)
    code, dev, T, E, pl = _logits(logits, K)
    pm = None if mask is None else _arg(mask, "mask", torch.bool, dev, (T,))
    if out is None:
        ids = torch.empty((T, K), dtype=torch.int32, device=dev)
        weights = torch.empty((T, K), dtype=torch.float32, device=dev)
        out = ExpertRoute(ids, weights, ids.new_empty(E), weights.new_empty(E), weights.new_empty(()),
                          ids.new_empty(1))
        po = [t.data_ptr() for t in (out.ids, out.weights, out.counts, out.shares, out.loss, out.kept)]
    else:
        po = [_arg(out.ids, "ids", torch.int32, dev, (T, K)), _arg(out.weights, "weights", torch.float32, dev, (T, K)),
              _arg(out.counts, "counts", torch.int32, dev, (E,)), _arg(out.shares, "shares", torch.float32, dev, (E,)),
              _arg(out.loss, "loss", torch.float32, dev, ()), _arg(out.kept, "kept", torch.int32, dev, (1,))]
    ws, pws, room = _room(lib.gs_expert_route_workspace_bytes(T, E), dev) if workspace is None \
        else _given_room(workspace, dev)
    _check(lib.gs_expert_route(pl, pm, T, E, K, int(bool(renormalize)), code, *po, pws, room, _stream_int(stream, dev)))
    return out


@_stream_scoped
def gs_expert_route_bwd(logits, route, grad_weights=None, grad_loss=None, renormalize=True, out=None, stream=None):
    """Gradient of sum(grad_weights * weights) + grad_loss * loss for the logits of gs_expert_route, in their type.
    grad_weights [tokens, choices] and grad_loss [] float32 (None: zero); renormalize as the forward's."""
    lib = load_library()
    K = route.ids.shape[1] if route.ids.dim() == 2 else 0
    code, dev, T, E, pl = _logits(logits, K)
    pi, pw = _arg(route.ids, "ids", torch.int32, dev, (T, K)), _arg(route.weights, "weights", torch.float32, dev, (T, K))
    pc, pk = _arg(route.counts, "counts", torch.int32, dev, (E,)), _arg(route.kept, "kept", torch.int32, dev, (1,))
    pg = None if grad_weights is None else _arg(grad_weights, "grad_weights", torch.float32, dev, (T, K))
    ps = None if grad_loss is None else _arg(grad_loss, "grad_loss", torch.float32, dev, ())
    if out is None:
        out = torch.empty_like(logits)
    else:
        _arg(out, "grad_logits", logits.dtype, dev, (T, E))
    _check(lib.gs_expert_route_bwd(pl, pi, pw, pc, pk, pg, ps, T, E, K, int(bool(renormalize)), code, out.data_ptr(),
                                   _stream_int(stream, dev)))
    return out


# ----------------------------------------------------------------------------------------------------------------
# Values held in 8 bits, and the experts' products of them


@dataclass
class Quantized:
    values: torch.Tensor  # [..., rows, blocks * 128] float8_e4m3fn, zeros past a row's end
    scales: torch.Tensor  # [..., rows, blocks] uint8: b stands for 2^(b - 127)
    dim: int  # values of a row


def _held(q, name, device=None):
    """(device, shape without the last axis, dim, address of the values, address of the scales) of a Quantized."""
    if not isinstance(q, Quantized):
        raise TypeError(f"{name} must be a Quantized (as gs_quantize gives)")
    if not isinstance(q.values, torch.Tensor):
        raise TypeError(f"{name} values must be a torch.Tensor")
    lead, dim = tuple(q.values.shape[:-1]), int(q.dim)
    if dim < 1:
        raise ValueError(f"{name} must have at least one column")
    blocks, dev = (dim + 127) // 128, q.values.device if device is None else device
    if not isinstance(q.scales, torch.Tensor) or tuple(q.scales.shape) != lead + (blocks,):
        raise ValueError(f"{name} scales must have shape {lead + (blocks,)}")
    pv = _arg(q.values, f"{name} values", torch.float8_e4m3fn, dev, lead + (blocks * 128,))
    return dev, lead, dim, pv, _arg(q.scales, f"{name} scales", torch.uint8, dev, lead + (blocks,))


@_stream_scoped
def gs_quantize(x, transpose=False, out=None, stream=None) -> Quantized:
    """x [..., rows, dim] (float32, bfloat16 or float16) held in 8 bits: e4m3 with a power of two for each block of 128
    along a row. transpose=True: of the transposed matrices, [..., dim, rows]."""
    lib = load_library()
    code, dev = _element(x, "x"), x.device
    if x.dim() < (2 if transpose else 1) or x.shape[-1] < 1:
        raise ValueError(f"x must be [{'..., rows' if transpose else '...'}, dim] (got {tuple(x.shape)})")
    px, dim = _arg(x, "x", x.dtype, dev, x.shape), x.shape[-1]
    if transpose:
        rows, lead, along = x.shape[-2], x.shape[:-2] + (dim,), x.shape[-2]
        if rows < 1:
            raise ValueError("x must have at least one row to transpose")
        batch = x.numel() // (rows * dim)
    else:
        batch, rows, lead, along = 1, x.numel() // dim, x.shape[:-1], dim
    blocks = (along + 127) // 128
    if out is None:
        out = Quantized(torch.empty(lead + (blocks * 128,), dtype=torch.float8_e4m3fn, device=dev),
                        torch.empty(lead + (blocks,), dtype=torch.uint8, device=dev), along)
        pv, ps = out.values.data_ptr(), out.scales.data_ptr()
    else:
        _, got, got_dim, pv, ps = _held(out, "out", dev)
        if got != tuple(lead) or got_dim != along:
            raise ValueError(f"out must hold {tuple(lead) + (along,)} (got {got + (got_dim,)})")
    _check(lib.gs_quantize(px, batch, rows, dim, int(bool(transpose)), code, pv, ps, _stream_int(stream, dev)))
    return out


@_stream_scoped
def gs_dequantize(q, dtype=torch.float32, out=None, stream=None):
    """The values that q stands for, [..., dim] of dtype (float32, bfloat16 or float16)."""
    lib = load_library()
    dev, lead, dim, pv, ps = _held(q, "q")
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be float32, bfloat16 or float16 (got {dtype})")
    if out is None:
        out = torch.empty(lead + (dim,), dtype=dtype, device=dev)
    else:
        _arg(out, "out", dtype, dev, lead + (dim,))
    _check(lib.gs_dequantize(pv, ps, q.scales.numel() // q.scales.shape[-1], dim, _DTYPES[dtype], out.data_ptr(),
                                _stream_int(stream, dev)))
    return out


def _plan_rows(lead, plan, gather, device):
    """(rows, x_rows, choices, experts, address of offsets, address of pairs) of x's rows under a plan."""
    if len(lead) != 1:
        raise ValueError("x must be [rows, dim]")
    n = lead[0]
    if plan is None:
        if gather:
            raise ValueError("gather needs a plan")
        return n, n, 1, 1, None, None
    T, K, E, po, _ = _plan_inputs(plan, device)
    if n != (T if gather else T * K):
        raise ValueError(f"x must have {T if gather else T * K} rows (got {n})")
    pp = _arg(plan.pairs, "pairs", torch.int32, device, (T * K,)) if gather else None
    return T * K, n, K, E, po, pp


@_stream_scoped
def gs_expert_product(x, weight, plan=None, gather=False, relu=False, dtype=torch.bfloat16, out=None, stream=None):
    """Every expert's rows times its weight: out[r] = x[r] @ weight[e(r)].T, [rows, cols] of dtype, zeros in the rows past
    the plan's kept ones; relu=True: max(0, .).

    x: Quantized rows in the plan's order, [tokens * choices, dim], or with gather=True the tokens themselves,
    [tokens, dim]. weight: Quantized [experts, cols, dim]. plan=None: one weight [cols, dim] for all rows. float32 results
    are summed in float32; for 16-bit ones the products of each 8 neighbours along dim are first cut off 2^-13 below the
    largest of them, so that results of large products that cancel keep fewer bits."""
    lib = load_library()
    dev, lead, dim, px, pxs = _held(x, "x")
    rows, x_rows, K, E, po, pp = _plan_rows(lead, plan, gather, dev)
    _, wide, wdim, pw, pws = _held(weight, "weight", dev)
    if wdim != dim or len(wide) != (1 if plan is None else 2) or wide[-1] < 1 or (plan is not None and wide[0] != E):
        raise ValueError(f"weight must hold [{'' if plan is None else f'{E}, '}cols, {dim}] (got {wide + (wdim,)})")
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be float32, bfloat16 or float16 (got {dtype})")
    cols = wide[-1]
    if out is None:
        out = torch.empty((rows, cols), dtype=dtype, device=dev)
    else:
        _arg(out, "out", dtype, dev, (rows, cols))
    _check(lib.gs_expert_product(px, pxs, pw, pws, po, pp, rows, x_rows, K, E, dim, cols, int(bool(relu)),
                                    _DTYPES[dtype], out.data_ptr(), _stream_int(stream, dev)))
    return out


@_stream_scoped
def gs_expert_weight_grad(x, grad, plan=None, gather=False, out=None, stream=None, workspace=None):
    """Every expert's weight gradient, x[rows of e].T @ grad[rows of e]: [experts, dim, cols] float32 ([dim, cols] without
    a plan). x as in gs_expert_product, grad [rows, cols] of float32, bfloat16 or float16; its rows past the plan's
    kept ones are not read."""
    lib = load_library()
    dev, lead, dim, px, pxs = _held(x, "x")
    rows, x_rows, K, E, po, pp = _plan_rows(lead, plan, gather, dev)
    code = _element(grad, "grad")
    if grad.dim() != 2 or grad.shape[0] != rows or grad.shape[1] < 1:
        raise ValueError(f"grad must be [{rows}, cols] (got {tuple(grad.shape)})")
    pg, cols = _arg(grad, "grad", grad.dtype, dev, grad.shape), grad.shape[1]
    shape = (dim, cols) if plan is None else (E, dim, cols)
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        _arg(out, "out", torch.float32, dev, shape)
    ws, pws, room = _room(lib.gs_expert_weight_grad_workspace_bytes(rows, E, dim, cols), dev) if workspace is None \
        else _given_room(workspace, dev)
    _check(lib.gs_expert_weight_grad(px, pxs, pg, po, pp, rows, x_rows, K, E, dim, cols, code, out.data_ptr(), pws,
                                        room, _stream_int(stream, dev)))
    return out
