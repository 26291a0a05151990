"""Thin Python binding of libgsa (include/gsa.h): argument marshalling only.

Functions with the C names (``grouped_scaled_act_fwd``, ``grouped_scaled_act_bwd``,
``gsa_layout``, ``gsa_workspace_size``, ``gsa_workspace_status``) take raw
pointers/ints exactly like the C ABI.  ``fwd`` / ``bwd`` are conveniences that
allocate output tensors with PyTorch (device memory is PyTorch's job here) and
call the C functions; every step of the computation runs in the CUDA kernel.
There is no fallback: if libgsa.so is missing or cannot load, this module
raises.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgsa.so")

ACT = {"srelu": 0, "tanh_srelu": 1, "swiglu": 2, "clamped_swiglu": 3, "gelu": 4, "sigmoid": 5, "identity": 6}
GLU_ACTS = (2, 3)
MXFP8, NVFP4 = 0, 1
SCALES_COMPACT, SCALES_TILED = 0, 1
STATUS = {0: "GSA_OK", 1: "GSA_ERR_INVALID_ARG", 2: "GSA_ERR_UNSUPPORTED", 3: "GSA_ERR_ALIGNMENT",
          4: "GSA_ERR_WORKSPACE", 5: "GSA_ERR_CUDA", 6: "GSA_ERR_DEVICE_TIMEOUT"}

EXPORTED = ["gsa_layout", "gsa_workspace_size", "grouped_scaled_act_fwd", "grouped_scaled_act_bwd",
            "gsa_workspace_status", "gsa_last_launch_count", "gsa_status_string", "gsa_version",
            "gsa_fwd_noalloc", "gsa_fwd_noalloc_status", "gsa_layout_bound", "gsa_workspace_size_graph_safe",
            "grouped_scaled_act_fwd_graph_safe", "grouped_scaled_act_bwd_graph_safe", "gsa_selftest_wait_timeout",
            "gsa_layout_ex", "gsa_layout_bound_ex", "gsa_moe_sort_workspace_size", "gsa_moe_sort", "gsa_moe_permute",
            "gsa_moe_permute_bwd", "gsa_moe_unpermute", "gsa_moe_unpermute_bwd", "gsa_grouped_gemm",
            "gsa_grouped_gemm_wgrad", "gsa_grouped_gemm_wgrad_workspace_size",
            "gsa_grouped_gemm_status", "gsa_grouped_glu", "gsa_grouped_glu_bwd", "gsa_grouped_glu_bwd_workspace_size",
            "gsa_grouped_gemv", "gsa_grouped_gemv_workspace_size", "gsa_grouped_glu_gemv"]


class GsaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class ActParams(ctypes.Structure):
    _fields_ = [("s", ctypes.c_float), ("limit", ctypes.c_float), ("alpha", ctypes.c_float),
                ("glu_linear_offset", ctypes.c_float)]


class Recipe(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("rht_colwise", ctypes.c_int32), ("rht_sign_mask", ctypes.c_uint32),
                ("scale_layout", ctypes.c_int32)]


class QOut(ctypes.Structure):
    _fields_ = [("row_data", ctypes.c_void_p), ("row_scale", ctypes.c_void_p), ("col_data", ctypes.c_void_p),
                ("col_scale", ctypes.c_void_p), ("amax_row", ctypes.c_void_p), ("amax_col", ctypes.c_void_p)]


class QIn(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("amax", ctypes.c_void_p),
                ("data_bytes", ctypes.c_int64), ("scale_bytes", ctypes.c_int64)]


class LayoutInfo(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("row_data_bytes", ctypes.c_int64), ("row_scale_bytes", ctypes.c_int64),
                ("col_data_bytes", ctypes.c_int64), ("col_scale_bytes", ctypes.c_int64),
                ("amax_floats", ctypes.c_int64)]


_lib = None
_P = ctypes.c_void_p
_I64 = ctypes.c_int64


def load():
    """Load libgsa.so (building it first if only the sources are present)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            from . import build
            build.build()
        L = ctypes.CDLL(LIB_PATH)
        L.gsa_layout.restype = ctypes.c_int
        L.gsa_layout.argtypes = [_I64, _P, _I64, ctypes.c_int32, ctypes.POINTER(LayoutInfo), _P, _P]
        L.gsa_workspace_size.restype = ctypes.c_size_t
        L.gsa_workspace_size.argtypes = [_I64, _P, _I64, ctypes.c_int32, ctypes.c_int32]
        L.grouped_scaled_act_fwd.restype = ctypes.c_int
        L.grouped_scaled_act_fwd.argtypes = [_P, _P, _P, _I64, _I64, ctypes.c_int32, ctypes.POINTER(ActParams),
                                             ctypes.POINTER(Recipe), ctypes.POINTER(QOut), _P, _P, ctypes.c_size_t, _P]
        L.grouped_scaled_act_bwd.restype = ctypes.c_int
        L.grouped_scaled_act_bwd.argtypes = [_P, _P, _P, _P, _I64, _I64, ctypes.c_int32, ctypes.POINTER(ActParams),
                                             ctypes.POINTER(Recipe), _P, ctypes.POINTER(QOut), _P,
                                             ctypes.POINTER(QOut), _P, ctypes.c_size_t, _P]
        L.gsa_fwd_noalloc.restype = ctypes.c_int
        L.gsa_fwd_noalloc.argtypes = [_P, _P, _P, _I64, _I64, ctypes.c_int32, ctypes.POINTER(ActParams),
                                      ctypes.POINTER(Recipe), ctypes.POINTER(QOut), _P, _P]
        L.gsa_fwd_noalloc_status.restype = ctypes.c_int
        L.gsa_fwd_noalloc_status.argtypes = [_P]
        L.gsa_layout_ex.restype = ctypes.c_int
        L.gsa_layout_ex.argtypes = [_I64, _P, _I64, ctypes.POINTER(Recipe), ctypes.POINTER(LayoutInfo), _P, _P, _P]
        L.gsa_layout_bound_ex.restype = ctypes.c_int
        L.gsa_layout_bound_ex.argtypes = [_I64, _I64, _I64, ctypes.POINTER(Recipe), ctypes.POINTER(LayoutInfo)]
        L.gsa_layout_bound.restype = ctypes.c_int
        L.gsa_layout_bound.argtypes = [_I64, _I64, _I64, ctypes.c_int32, ctypes.POINTER(LayoutInfo)]
        L.gsa_workspace_size_graph_safe.restype = ctypes.c_size_t
        L.gsa_workspace_size_graph_safe.argtypes = [_I64, _I64, _I64, ctypes.c_int32, ctypes.c_int32]
        L.grouped_scaled_act_fwd_graph_safe.restype = ctypes.c_int
        L.grouped_scaled_act_fwd_graph_safe.argtypes = [_P, _P, _P, _I64, _I64, _I64, ctypes.c_int32,
                                                        ctypes.POINTER(ActParams), ctypes.POINTER(Recipe),
                                                        ctypes.POINTER(QOut), _P, _P, _P, ctypes.c_size_t, _P]
        L.grouped_scaled_act_bwd_graph_safe.restype = ctypes.c_int
        L.grouped_scaled_act_bwd_graph_safe.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_int32,
                                                        ctypes.POINTER(ActParams), ctypes.POINTER(Recipe), _P,
                                                        ctypes.POINTER(QOut), _P, ctypes.POINTER(QOut), _P, _P,
                                                        ctypes.c_size_t, _P]
        L.gsa_selftest_wait_timeout.restype = ctypes.c_int
        L.gsa_selftest_wait_timeout.argtypes = [_P, ctypes.c_int32, ctypes.c_uint32, _P]
        L.gsa_workspace_status.restype = ctypes.c_int
        L.gsa_workspace_status.argtypes = [_P, _P]
        L.gsa_last_launch_count.restype = ctypes.c_int32
        L.gsa_last_launch_count.argtypes = []
        L.gsa_status_string.restype = ctypes.c_char_p
        L.gsa_status_string.argtypes = [ctypes.c_int]
        route = [_I64, _I64, _I64, ctypes.c_int32]   # tokens, topk, hidden, dtype
        for name, args in (("gsa_moe_sort", [_P, ctypes.c_int32, _I64, _I64, _I64, _P, _P, _P, ctypes.c_size_t, _P]),
                           ("gsa_moe_permute", [_P, _P, _P, *route, _P, _P, _P]),
                           ("gsa_moe_permute_bwd", [_P, _P, _P, *route, _P, _P, _P]),
                           ("gsa_moe_unpermute", [_P, _P, _P, *route, _P, _P]),
                           ("gsa_moe_unpermute_bwd", [_P, _P, _P, _P, *route, _P, _P, _P])):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = args
        L.gsa_moe_sort_workspace_size.restype = ctypes.c_size_t
        L.gsa_moe_sort_workspace_size.argtypes = [_I64, _I64, _I64]
        L.gsa_grouped_gemm.restype = ctypes.c_int
        L.gsa_grouped_gemm.argtypes = [ctypes.POINTER(QIn), ctypes.POINTER(QIn), _P, _I64, _I64, _I64, _I64,
                                       ctypes.c_int32, _P, ctypes.c_int32, _P]
        L.gsa_grouped_gemm_wgrad.restype = ctypes.c_int
        L.gsa_grouped_gemm_wgrad.argtypes = [ctypes.POINTER(QIn), ctypes.POINTER(QIn), _P, _I64, _I64, _I64, _I64,
                                             ctypes.c_int32, _P, ctypes.c_int32, ctypes.c_int32, _P,
                                             ctypes.c_size_t, _P]
        L.gsa_grouped_gemm_wgrad_workspace_size.restype = ctypes.c_size_t
        L.gsa_grouped_gemm_wgrad_workspace_size.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int32]
        L.gsa_grouped_gemm_status.restype = ctypes.c_int
        L.gsa_grouped_gemm_status.argtypes = [_P]
        i32, q = ctypes.c_int32, ctypes.POINTER(QIn)
        shape = [_P, _I64, _I64, _I64, _I64, i32]                     # split, E, M, N, K, recipe
        gated = [i32, ctypes.POINTER(ActParams), _P, i32]             # activation, its parameters, probs, b_groups
        for name, args in (("gsa_grouped_glu", [q, q, *shape, *gated, _P, i32, _P]),
                           ("gsa_grouped_glu_bwd", [_P, q, q, *shape, *gated, _P, i32, _P, _P, ctypes.c_size_t, _P]),
                           ("gsa_grouped_gemv", [_P, i32, q, *shape, _P, i32, _P, ctypes.c_size_t, _P]),
                           ("gsa_grouped_glu_gemv", [_P, i32, q, *shape, *gated, _P, i32, _P, ctypes.c_size_t, _P])):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = args
        L.gsa_grouped_gemv_workspace_size.restype = ctypes.c_size_t
        L.gsa_grouped_gemv_workspace_size.argtypes = [_I64, _I64, _I64, i32]
        L.gsa_grouped_glu_bwd_workspace_size.restype = ctypes.c_size_t
        L.gsa_grouped_glu_bwd_workspace_size.argtypes = [_I64, _I64]
        L.gsa_version.restype = ctypes.c_int32
        L.gsa_version.argtypes = []
        _lib = L
    return _lib


# ------------------------------------------------------------ C-named calls

def _split_array(split_sizes):
    arr = (ctypes.c_int64 * len(split_sizes))(*[int(s) for s in split_sizes])
    return arr


def gsa_layout(split_sizes, width: int, recipe_kind: int):
    """-> (LayoutInfo, col_data_offsets[E+1], col_scale_offsets[E+1])."""
    E = len(split_sizes)
    info = LayoutInfo()
    d = (ctypes.c_int64 * (E + 1))()
    s = (ctypes.c_int64 * (E + 1))()
    st = load().gsa_layout(E, ctypes.cast(_split_array(split_sizes), _P), int(width), int(recipe_kind),
                           ctypes.byref(info), ctypes.cast(d, _P), ctypes.cast(s, _P))
    if st != 0:
        raise GsaError(st, "gsa_layout")
    return info, list(d), list(s)


def gsa_layout_ex(split_sizes, width: int, recipe: Recipe):
    """-> (LayoutInfo, col_data_offsets[E+1], col_scale_offsets[E+1], row_scale_offsets[E+1])."""
    E = len(split_sizes)
    info = LayoutInfo()
    d = (ctypes.c_int64 * (E + 1))()
    s = (ctypes.c_int64 * (E + 1))()
    r = (ctypes.c_int64 * (E + 1))()
    st = load().gsa_layout_ex(E, ctypes.cast(_split_array(split_sizes), _P), int(width), ctypes.byref(recipe),
                              ctypes.byref(info), ctypes.cast(d, _P), ctypes.cast(s, _P), ctypes.cast(r, _P))
    if st != 0:
        raise GsaError(st, "gsa_layout_ex")
    return info, list(d), list(s), list(r)


def gsa_layout_bound_ex(E: int, M: int, width: int, recipe: Recipe) -> LayoutInfo:
    info = LayoutInfo()
    st = load().gsa_layout_bound_ex(int(E), int(M), int(width), ctypes.byref(recipe), ctypes.byref(info))
    if st != 0:
        raise GsaError(st, "gsa_layout_bound_ex")
    return info


def gsa_workspace_size(split_sizes, w_in: int, act_kind: int, recipe_kind: int) -> int:
    return int(load().gsa_workspace_size(len(split_sizes), ctypes.cast(_split_array(split_sizes), _P), int(w_in),
                                         int(act_kind), int(recipe_kind)))


def grouped_scaled_act_fwd(x_ptr, probs_ptr, split_sizes, w_in, act_kind, act_params: ActParams, recipe: Recipe,
                           y_q: QOut, y_bf16_ptr, ws_ptr, ws_bytes, stream_ptr) -> int:
    return load().grouped_scaled_act_fwd(x_ptr, probs_ptr, ctypes.cast(_split_array(split_sizes), _P),
                                         len(split_sizes), int(w_in), int(act_kind), ctypes.byref(act_params),
                                         ctypes.byref(recipe), ctypes.byref(y_q) if y_q is not None else None,
                                         y_bf16_ptr, ws_ptr, int(ws_bytes), stream_ptr)


def grouped_scaled_act_bwd(dy_ptr, x_ptr, probs_ptr, split_sizes, w_in, act_kind, act_params: ActParams,
                           recipe: Recipe, dx_bf16_ptr, dx_q: QOut | None, dprobs_ptr, y_regen: QOut | None,
                           ws_ptr, ws_bytes, stream_ptr) -> int:
    return load().grouped_scaled_act_bwd(dy_ptr, x_ptr, probs_ptr, ctypes.cast(_split_array(split_sizes), _P),
                                         len(split_sizes), int(w_in), int(act_kind), ctypes.byref(act_params),
                                         ctypes.byref(recipe), dx_bf16_ptr,
                                         ctypes.byref(dx_q) if dx_q is not None else None, dprobs_ptr,
                                         ctypes.byref(y_regen) if y_regen is not None else None,
                                         ws_ptr, int(ws_bytes), stream_ptr)


def gsa_fwd_noalloc(x_ptr, probs_ptr, split_sizes, w_in, act_kind, act_params: ActParams, recipe: Recipe,
                    y_q: QOut, y_bf16_ptr, stream_ptr) -> int:
    """Forward with the library's own fixed scratch instead of a workspace (no allocation)."""
    return load().gsa_fwd_noalloc(x_ptr, probs_ptr, ctypes.cast(_split_array(split_sizes), _P), len(split_sizes),
                                  int(w_in), int(act_kind), ctypes.byref(act_params), ctypes.byref(recipe),
                                  ctypes.byref(y_q) if y_q is not None else None, y_bf16_ptr, stream_ptr)


def gsa_fwd_noalloc_status(stream_ptr) -> int:
    """Error word of the last gsa_fwd_noalloc call on the current device (synchronizes the stream)."""
    return load().gsa_fwd_noalloc_status(stream_ptr)


def gsa_layout_bound(E: int, M: int, width: int, recipe_kind: int) -> LayoutInfo:
    """Sizes of the quantized copies for any split of M rows over E experts."""
    info = LayoutInfo()
    st = load().gsa_layout_bound(int(E), int(M), int(width), int(recipe_kind), ctypes.byref(info))
    if st != 0:
        raise GsaError(st, "gsa_layout_bound")
    return info


def gsa_workspace_size_graph_safe(E: int, M: int, w_in: int, act_kind: int, recipe_kind: int) -> int:
    return int(load().gsa_workspace_size_graph_safe(int(E), int(M), int(w_in), int(act_kind), int(recipe_kind)))


def grouped_scaled_act_fwd_graph_safe(x_ptr, probs_ptr, split_dev_ptr, E, M, w_in, act_kind, act_params: ActParams,
                                      recipe: Recipe, y_q: QOut, y_bf16_ptr, pad_ptr, ws_ptr, ws_bytes,
                                      stream_ptr) -> int:
    return load().grouped_scaled_act_fwd_graph_safe(x_ptr, probs_ptr, split_dev_ptr, int(E), int(M), int(w_in),
                                                    int(act_kind), ctypes.byref(act_params), ctypes.byref(recipe),
                                                    ctypes.byref(y_q) if y_q is not None else None, y_bf16_ptr,
                                                    pad_ptr, ws_ptr, int(ws_bytes), stream_ptr)


def grouped_scaled_act_bwd_graph_safe(dy_ptr, x_ptr, probs_ptr, split_dev_ptr, E, M, w_in, act_kind,
                                      act_params: ActParams, recipe: Recipe, dx_bf16_ptr, dx_q: QOut | None,
                                      dprobs_ptr, y_regen: QOut | None, pad_ptr, ws_ptr, ws_bytes, stream_ptr) -> int:
    return load().grouped_scaled_act_bwd_graph_safe(dy_ptr, x_ptr, probs_ptr, split_dev_ptr, int(E), int(M),
                                                    int(w_in), int(act_kind), ctypes.byref(act_params),
                                                    ctypes.byref(recipe), dx_bf16_ptr,
                                                    ctypes.byref(dx_q) if dx_q is not None else None, dprobs_ptr,
                                                    ctypes.byref(y_regen) if y_regen is not None else None,
                                                    pad_ptr, ws_ptr, int(ws_bytes), stream_ptr)


def gsa_selftest_wait_timeout(ws_ptr, which: int, limit_ms: int, stream_ptr) -> int:
    """Run a bounded wait that nothing signals (0: counter, 1: mbarrier) with a short limit."""
    return load().gsa_selftest_wait_timeout(ws_ptr, int(which), int(limit_ms), stream_ptr)


def gsa_workspace_status(ws_ptr, stream_ptr) -> int:
    return load().gsa_workspace_status(ws_ptr, stream_ptr)


def gsa_last_launch_count() -> int:
    return int(load().gsa_last_launch_count())


# ------------------------------------------------------- torch conveniences

def act_params(act: str | int, s: float = 4.0, limit: float = 7.0, alpha: float = 1.702,
               glu_linear_offset: float = 1.0) -> ActParams:
    return ActParams(s, limit, alpha, glu_linear_offset)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _record_layout(out: dict, scale_layout: int, keys=("row_scale", "col_scale")) -> None:
    """Notes on the scale buffers the layout they are written in: the products take tiled scales only, and the byte
    counts of both layouts are often the same."""
    for k in keys:
        if k in out:
            out[k].scale_layout = scale_layout


def alloc_qtensor(split_sizes, width: int, recipe_kind: int, rowwise: bool, columnwise: bool, device,
                  amax_experts: int | None = None, scale_layout: int = SCALES_COMPACT) -> dict:
    """Allocate the quantized copies of a [M, width] grouped tensor (uint8).
    Tiled scales are zero-filled (the library does not write their padding)."""
    import torch
    info = gsa_layout_ex(split_sizes, width, Recipe(recipe_kind, 0, 0, scale_layout))[0]
    E = len(split_sizes)
    sbuf = torch.zeros if scale_layout == SCALES_TILED else torch.empty
    out = {}
    if rowwise:
        out["row_data"] = torch.empty(max(1, info.row_data_bytes), dtype=torch.uint8, device=device)
        out["row_scale"] = sbuf(max(1, info.row_scale_bytes), dtype=torch.uint8, device=device)
    if columnwise:
        out["col_data"] = torch.empty(max(1, info.col_data_bytes), dtype=torch.uint8, device=device)
        out["col_scale"] = sbuf(max(1, info.col_scale_bytes), dtype=torch.uint8, device=device)
    if recipe_kind == NVFP4:
        if rowwise:
            out["amax_row"] = torch.empty(E, dtype=torch.float32, device=device)
        if columnwise:
            out["amax_col"] = torch.empty(E, dtype=torch.float32, device=device)
    out["_info"] = info
    _record_layout(out, scale_layout)
    return out


def qout_of(q: dict | None) -> QOut | None:
    if q is None:
        return None
    return QOut(*[(q[k].data_ptr() if k in q else None) for k in
                  ("row_data", "row_scale", "col_data", "col_scale", "amax_row", "amax_col")])


class Workspace:
    """A device workspace sized by gsa_workspace_size (256-byte aligned)."""

    def __init__(self, split_sizes, w_in, act_kind, recipe_kind, device):
        import torch
        self.nbytes = gsa_workspace_size(split_sizes, w_in, act_kind, recipe_kind)
        if self.nbytes == 0:
            raise GsaError(1, "gsa_workspace_size")
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        base = self.buf.data_ptr()
        self.ptr = (base + 255) // 256 * 256

    def status(self, stream=None) -> int:
        return gsa_workspace_status(ctypes.c_void_p(self.ptr), _stream_ptr(stream))


def _check(st, what):
    if st != 0:
        raise GsaError(st, what)


def fwd(x, probs, split_sizes, act: str, recipe_kind: int, rht: bool = False, rht_mask: int = 0,
        rowwise: bool = True, columnwise: bool = True, want_y: bool = False, params: ActParams | None = None,
        ws: Workspace | None = None, out: dict | None = None, stream=None, scale_layout: int = SCALES_COMPACT) -> dict:
    """Forward on device tensors x [M, W_in] bf16, probs [M] f32 (or None: p = 1).  Returns a dict
    with the quantized copies (row_data, row_scale, col_data, col_scale,
    amax_row, amax_col) and, with want_y, the BF16 Y."""
    import torch
    a = ACT[act] if isinstance(act, str) else int(act)
    w_in = x.shape[1]
    w = w_in // 2 if a in GLU_ACTS else w_in
    params = params or act_params(a)
    ws = ws or Workspace(split_sizes, w_in, a, recipe_kind, x.device)
    if out is None:
        out = alloc_qtensor(split_sizes, w, recipe_kind, rowwise, columnwise, x.device, scale_layout=scale_layout)
        if want_y:
            out["y"] = torch.empty((x.shape[0], w), dtype=torch.bfloat16, device=x.device)
    rec = Recipe(recipe_kind, int(bool(rht)), int(rht_mask) & 0xFFFF, scale_layout)
    st = grouped_scaled_act_fwd(_ptr(x), _ptr(probs), split_sizes, w_in, a, params, rec, qout_of(out),
                                _ptr(out.get("y")), ctypes.c_void_p(ws.ptr), ws.nbytes, _stream_ptr(stream))
    _check(st, "grouped_scaled_act_fwd")
    _record_layout(out, scale_layout)
    return out


def bwd(dy, x, probs, split_sizes, act: str, recipe_kind: int, rht: bool = False, rht_mask: int = 0,
        want_dx: bool = True, rowwise: bool = True, columnwise: bool = True, want_dprobs: bool = True,
        regen: bool = False, params: ActParams | None = None, ws: Workspace | None = None,
        out: dict | None = None, stream=None, scale_layout: int = SCALES_COMPACT) -> dict:
    """Backward on device tensors.  Returns dx (bf16 [M, W_in]), dprobs (f32 [M]),
    the quantized copies of dX and, with regen, the regenerated columnwise copy
    of Y under keys prefixed 'y_'."""
    import torch
    a = ACT[act] if isinstance(act, str) else int(act)
    w_in = x.shape[1]
    w = w_in // 2 if a in GLU_ACTS else w_in
    params = params or act_params(a)
    ws = ws or Workspace(split_sizes, w_in, a, recipe_kind, x.device)
    if out is None:
        out = {}
        if rowwise or columnwise:
            out.update(alloc_qtensor(split_sizes, w_in, recipe_kind, rowwise, columnwise, x.device,
                                     scale_layout=scale_layout))
        if want_dx:
            out["dx"] = torch.empty((x.shape[0], w_in), dtype=torch.bfloat16, device=x.device)
        if want_dprobs:
            out["dprobs"] = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        if regen:
            yq = alloc_qtensor(split_sizes, w, recipe_kind, False, True, x.device, scale_layout=scale_layout)
            for k, v in yq.items():
                out["y_" + k] = v
    dxq = qout_of({k: v for k, v in out.items() if not k.startswith("y_") and k not in ("dx", "dprobs", "_info")}) \
        if (rowwise or columnwise) else None
    yq = qout_of({k[2:]: v for k, v in out.items() if k.startswith("y_") and k != "y__info"}) if regen else None
    rec = Recipe(recipe_kind, int(bool(rht)), int(rht_mask) & 0xFFFF, scale_layout)
    st = grouped_scaled_act_bwd(_ptr(dy), _ptr(x), _ptr(probs), split_sizes, w_in, a, params, rec,
                                _ptr(out.get("dx")), dxq, _ptr(out.get("dprobs")), yq,
                                ctypes.c_void_p(ws.ptr), ws.nbytes, _stream_ptr(stream))
    _check(st, "grouped_scaled_act_bwd")
    _record_layout(out, scale_layout, (("row_scale", "col_scale") if dxq else ()) + (("y_col_scale",) if yq else ()))
    return out


# ------------------------------------------------- graph-safe conveniences

def alloc_qtensor_bound(E: int, M: int, width: int, recipe_kind: int, rowwise: bool, columnwise: bool,
                        device, scale_layout: int = SCALES_COMPACT) -> dict:
    """Quantized copies sized for any split of M rows over E experts."""
    import torch
    info = gsa_layout_bound_ex(E, M, width, Recipe(recipe_kind, 0, 0, scale_layout))
    sbuf = torch.zeros if scale_layout == SCALES_TILED else torch.empty
    out = {}
    if rowwise:
        out["row_data"] = torch.empty(max(1, info.row_data_bytes), dtype=torch.uint8, device=device)
        out["row_scale"] = sbuf(max(1, info.row_scale_bytes), dtype=torch.uint8, device=device)
    if columnwise:
        out["col_data"] = torch.empty(max(1, info.col_data_bytes), dtype=torch.uint8, device=device)
        out["col_scale"] = sbuf(max(1, info.col_scale_bytes), dtype=torch.uint8, device=device)
    if recipe_kind == NVFP4:
        if rowwise:
            out["amax_row"] = torch.empty(E, dtype=torch.float32, device=device)
        if columnwise:
            out["amax_col"] = torch.empty(E, dtype=torch.float32, device=device)
    out["_info"] = info
    _record_layout(out, scale_layout)
    return out


class GraphSafeWorkspace(Workspace):
    """Workspace of the graph-safe calls, sized by (E, M) alone."""

    def __init__(self, E, M, w_in, act_kind, recipe_kind, device):
        import torch
        self.nbytes = gsa_workspace_size_graph_safe(E, M, w_in, act_kind, recipe_kind)
        if self.nbytes == 0:
            raise GsaError(1, "gsa_workspace_size_graph_safe")
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        self.ptr = (self.buf.data_ptr() + 255) // 256 * 256


def fwd_graph_safe(x, probs, split_dev, act: str, recipe_kind: int, rht: bool = False, rht_mask: int = 0,
                   rowwise: bool = True, columnwise: bool = True, want_y: bool = False,
                   params: ActParams | None = None, ws: Workspace | None = None, out: dict | None = None,
                   stream=None, scale_layout: int = SCALES_COMPACT) -> dict:
    """Forward with split_dev ([E] int64 on the device).  Outputs sized by
    gsa_layout_bound; out["pad"] ([E+1] int64) receives the padded row
    offsets of the columnwise blocks.  Enqueues work only: capturable."""
    import torch
    a = ACT[act] if isinstance(act, str) else int(act)
    E, M, w_in = split_dev.numel(), x.shape[0], x.shape[1]
    w = w_in // 2 if a in GLU_ACTS else w_in
    params = params or act_params(a)
    ws = ws or GraphSafeWorkspace(E, M, w_in, a, recipe_kind, x.device)
    if out is None:
        out = alloc_qtensor_bound(E, M, w, recipe_kind, rowwise, columnwise, x.device, scale_layout)
        if want_y:
            out["y"] = torch.empty((M, w), dtype=torch.bfloat16, device=x.device)
        out["pad"] = torch.empty(E + 1, dtype=torch.int64, device=x.device)
    rec = Recipe(recipe_kind, int(bool(rht)), int(rht_mask) & 0xFFFF, scale_layout)
    st = grouped_scaled_act_fwd_graph_safe(_ptr(x), _ptr(probs), _ptr(split_dev), E, M, w_in, a, params, rec,
                                           qout_of(out), _ptr(out.get("y")), _ptr(out.get("pad")),
                                           ctypes.c_void_p(ws.ptr), ws.nbytes, _stream_ptr(stream))
    _check(st, "grouped_scaled_act_fwd_graph_safe")
    _record_layout(out, scale_layout)
    return out


def bwd_graph_safe(dy, x, probs, split_dev, act: str, recipe_kind: int, rht: bool = False, rht_mask: int = 0,
                   want_dx: bool = True, rowwise: bool = True, columnwise: bool = True, want_dprobs: bool = True,
                   regen: bool = False, params: ActParams | None = None, ws: Workspace | None = None,
                   out: dict | None = None, stream=None, scale_layout: int = SCALES_COMPACT) -> dict:
    """Backward with split_dev on the device; keys as for bwd, plus "pad"."""
    import torch
    a = ACT[act] if isinstance(act, str) else int(act)
    E, M, w_in = split_dev.numel(), x.shape[0], x.shape[1]
    w = w_in // 2 if a in GLU_ACTS else w_in
    params = params or act_params(a)
    ws = ws or GraphSafeWorkspace(E, M, w_in, a, recipe_kind, x.device)
    if out is None:
        out = {}
        if rowwise or columnwise:
            out.update(alloc_qtensor_bound(E, M, w_in, recipe_kind, rowwise, columnwise, x.device, scale_layout))
        if want_dx:
            out["dx"] = torch.empty((M, w_in), dtype=torch.bfloat16, device=x.device)
        if want_dprobs:
            out["dprobs"] = torch.empty(M, dtype=torch.float32, device=x.device)
        if regen:
            for k, v in alloc_qtensor_bound(E, M, w, recipe_kind, False, True, x.device, scale_layout).items():
                out["y_" + k] = v
        out["pad"] = torch.empty(E + 1, dtype=torch.int64, device=x.device)
    skip = ("dx", "dprobs", "_info", "pad")
    dxq = qout_of({k: v for k, v in out.items() if not k.startswith("y_") and k not in skip}) \
        if (rowwise or columnwise) else None
    yq = qout_of({k[2:]: v for k, v in out.items() if k.startswith("y_") and k != "y__info"}) if regen else None
    rec = Recipe(recipe_kind, int(bool(rht)), int(rht_mask) & 0xFFFF, scale_layout)
    st = grouped_scaled_act_bwd_graph_safe(_ptr(dy), _ptr(x), _ptr(probs), _ptr(split_dev), E, M, w_in, a, params,
                                           rec, _ptr(out.get("dx")), dxq, _ptr(out.get("dprobs")), yq,
                                           _ptr(out.get("pad")), ctypes.c_void_p(ws.ptr), ws.nbytes,
                                           _stream_ptr(stream))
    _check(st, "grouped_scaled_act_bwd_graph_safe")
    _record_layout(out, scale_layout, (("row_scale", "col_scale") if dxq else ()) + (("y_col_scale",) if yq else ()))
    return out


# ------------------------------------------- tokens into expert order and back
#
# Small calls are bound by the host, so the checks below are written to be cheap:
# no imports, no objects and no repeated lookups on the path of a good call.

BF16, FP16, FP32 = 0, 1, 2
_torch = None
_raw_stream = None
_current_device = None
_DTYPES: dict = {}


def _setup():
    """The torch module, imported on the first call, and the element type codes."""
    global _torch, _raw_stream, _current_device
    import torch
    _DTYPES.update({torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32})
    load()
    # the current stream's handle without a Stream object (2 us), where this torch has the call
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch
    return torch


def _refuse(t, what, shape, dtype):
    raise GsaError(1, f"{what}: contiguous CUDA {dtype} {list(shape)} expected, got {t.device} {t.dtype} "
                      f"{list(t.shape)}{'' if t.is_contiguous() else ' (not contiguous)'}")


def _require(t, what, shape, dtype):
    """A contiguous CUDA tensor of this shape and type."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _refuse(t, what, shape, dtype)


def _same_device(what, device, *tensors):
    for t in tensors:
        if t is not None and t.device != device:
            raise GsaError(1, f"{what}: tensors on {t.device} and {device}")


def _stream_of(stream, device, *inputs):
    """Handle of `stream`, or of the device's current one.  Inputs of a call on an explicit stream are recorded on
    it, so that the caching allocator keeps them until the stream is done with them.  The library launches on the
    current device (whose null stream a handle of 0 is), so tensors or a stream of another one are refused."""
    if device.index != _current_device():
        raise GsaError(1, f"tensors on {device}, but the current device is cuda:{_current_device()}")
    if stream is None:
        return _raw_stream(device.index)
    if stream.device != device:
        raise GsaError(1, f"tensors on {device}, stream of {stream.device}")
    for t in inputs:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


def _out(given, what, shape, dtype, device, stream):
    """The caller's output tensor, or a new one that belongs to the call's stream."""
    if given is not None:
        _require(given, what, shape, dtype)
        _same_device(what, device, given)
        if stream is not None:
            given.record_stream(stream)
        return given
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


def moe_sort(expert_idx, experts: int, out: tuple | None = None, stream=None):
    """Sort plan of expert_idx [tokens, topk] (int32 / int64; a value outside [0, experts) drops the slot):
    -> (row_of_slot [tokens, topk] int32, split_sizes [experts + 1] int64), both on the device."""
    torch = _torch or _setup()
    dt = expert_idx.dtype
    if (dt is not torch.int64 and dt is not torch.int32) or expert_idx.dim() != 2:
        raise GsaError(1, "moe_sort: expert_idx must be int32 or int64 [tokens, topk]")
    shape, dev = expert_idx.shape, expert_idx.device
    _require(expert_idx, "moe_sort: expert_idx", shape, dt)
    tokens, topk = shape
    row, split = out or (None, None)
    row = _out(row, "moe_sort: row_of_slot", shape, torch.int32, dev, stream)
    split = _out(split, "moe_sort: split_sizes", (max(0, experts) + 1,), torch.int64, dev, stream)
    nbytes = _lib.gsa_moe_sort_workspace_size(tokens, topk, experts)
    ws = _out(None, "", (nbytes,), torch.uint8, dev, stream) if nbytes else None
    st = _lib.gsa_moe_sort(expert_idx.data_ptr(), 8 if dt is torch.int64 else 4, tokens, topk, experts,
                           row.data_ptr(), split.data_ptr(), ws.data_ptr() if nbytes else None, nbytes,
                           _stream_of(stream, dev, expert_idx))
    if st:
        _check(st, "gsa_moe_sort")
    return row, split


MAX_GROUPS = 256


def moe_groups(split_sizes):
    """The groups of the sorted rows, from moe_sort's split_sizes [experts + 1]: that split itself, the dropped rows its
    last group.  With 256 experts, one group more than the graph-safe calls take: [256], the dropped rows counted to the
    last expert (rows of zeros behind its own, which change no result).  The first `experts` entries are the split of
    the products."""
    if split_sizes.shape[0] <= MAX_GROUPS:
        return split_sizes
    groups = split_sizes[:-1].clone()
    groups[-1:] += split_sizes[-1:]
    return groups


def _plan_and_rows(what, row_of_slot, rows, by_slot):
    """(tokens, topk, hidden, dtype code, device) of a plan and a [tokens or tokens * topk, hidden] row tensor."""
    torch = _torch or _setup()
    if row_of_slot.dim() != 2 or rows.dim() != 2:
        raise GsaError(1, f"{what}: row_of_slot [tokens, topk] and [rows, hidden] rows expected")
    tokens, topk = row_of_slot.shape
    _require(row_of_slot, what + ": row_of_slot", row_of_slot.shape, torch.int32)
    hidden = rows.shape[1]
    code = _DTYPES.get(rows.dtype)
    if code is None:
        raise GsaError(1, f"{what}: element type {rows.dtype} (bfloat16, float16 or float32 expected)")
    _require(rows, what + ": rows", (tokens * topk if by_slot else tokens, hidden), rows.dtype)
    dev = rows.device
    if row_of_slot.device != dev:
        _same_device(what, dev, row_of_slot)
    return tokens, topk, hidden, code, dev


def moe_permute(x, row_of_slot, probs=None, out: tuple | None = None, stream=None):
    """Token rows x [tokens, hidden] into expert order: xs [tokens * topk, hidden], and with probs
    [tokens, topk] (FP32) -> (xs, ps [tokens * topk])."""
    tokens, topk, hidden, code, dev = _plan_and_rows("moe_permute", row_of_slot, x, False)
    xs, ps = (out if probs is not None else (out, None)) if out is not None else (None, None)
    xs = _out(xs, "moe_permute: xs", (tokens * topk, hidden), x.dtype, dev, stream)
    pp = po = None
    if probs is not None:
        _require(probs, "moe_permute: probs", (tokens, topk), _torch.float32)
        _same_device("moe_permute", dev, probs)
        ps = _out(ps, "moe_permute: ps", (tokens * topk,), _torch.float32, dev, stream)
        pp, po = probs.data_ptr(), ps.data_ptr()
    st = _lib.gsa_moe_permute(x.data_ptr(), pp, row_of_slot.data_ptr(), tokens, topk, hidden, code, xs.data_ptr(), po,
                              _stream_of(stream, dev, x, row_of_slot, probs))
    if st:
        _check(st, "gsa_moe_permute")
    return xs if probs is None else (xs, ps)


def moe_permute_bwd(dxs, row_of_slot, dps=None, out: tuple | None = None, stream=None):
    """Gradient of moe_permute: dx [tokens, hidden], and with dps [tokens * topk] -> (dx, dprobs)."""
    tokens, topk, hidden, code, dev = _plan_and_rows("moe_permute_bwd", row_of_slot, dxs, True)
    dx, dprobs = (out if dps is not None else (out, None)) if out is not None else (None, None)
    dx = _out(dx, "moe_permute_bwd: dx", (tokens, hidden), dxs.dtype, dev, stream)
    pp = po = None
    if dps is not None:
        _require(dps, "moe_permute_bwd: dps", (tokens * topk,), _torch.float32)
        _same_device("moe_permute_bwd", dev, dps)
        dprobs = _out(dprobs, "moe_permute_bwd: dprobs", (tokens, topk), _torch.float32, dev, stream)
        pp, po = dps.data_ptr(), dprobs.data_ptr()
    st = _lib.gsa_moe_permute_bwd(dxs.data_ptr(), pp, row_of_slot.data_ptr(), tokens, topk, hidden, code,
                                  dx.data_ptr(), po, _stream_of(stream, dev, dxs, row_of_slot, dps))
    if st:
        _check(st, "gsa_moe_permute_bwd")
    return dx if dps is None else (dx, dprobs)


def _weights(what, weights, tokens, topk, dev):
    if weights is None:
        return None
    _require(weights, what + ": weights", (tokens, topk), _torch.float32)
    _same_device(what, dev, weights)
    return weights.data_ptr()


def moe_unpermute(ys, row_of_slot, weights=None, out=None, stream=None):
    """Expert rows ys [tokens * topk, hidden] back to tokens: out [tokens, hidden], the sum over a token's slots
    weighted by weights [tokens, topk] (FP32; None: 1)."""
    tokens, topk, hidden, code, dev = _plan_and_rows("moe_unpermute", row_of_slot, ys, True)
    wp = _weights("moe_unpermute", weights, tokens, topk, dev)
    out = _out(out, "moe_unpermute: out", (tokens, hidden), ys.dtype, dev, stream)
    st = _lib.gsa_moe_unpermute(ys.data_ptr(), wp, row_of_slot.data_ptr(), tokens, topk, hidden, code, out.data_ptr(),
                                _stream_of(stream, dev, ys, row_of_slot, weights))
    if st:
        _check(st, "gsa_moe_unpermute")
    return out


def moe_unpermute_bwd(dout, ys, row_of_slot, weights=None, want_dys: bool = True, out: tuple | None = None,
                      stream=None):
    """Gradient of moe_unpermute for dout [tokens, hidden]: (dys [tokens * topk, hidden], dweights [tokens, topk]
    FP32).  ys = None skips dweights, want_dys = False skips dys (None in its place)."""
    tokens, topk, hidden, code, dev = _plan_and_rows("moe_unpermute_bwd", row_of_slot, dout, False)
    wp = _weights("moe_unpermute_bwd", weights, tokens, topk, dev)
    dys, dw = out if out is not None else (None, None)
    if want_dys:
        dys = _out(dys, "moe_unpermute_bwd: dys", (tokens * topk, hidden), dout.dtype, dev, stream)
    if ys is not None:
        _require(ys, "moe_unpermute_bwd: ys", (tokens * topk, hidden), dout.dtype)
        _same_device("moe_unpermute_bwd", dev, ys)
        dw = _out(dw, "moe_unpermute_bwd: dweights", (tokens, topk), _torch.float32, dev, stream)
    st = _lib.gsa_moe_unpermute_bwd(dout.data_ptr(), None if ys is None else ys.data_ptr(), wp, row_of_slot.data_ptr(),
                                    tokens, topk, hidden, code, dys.data_ptr() if want_dys else None,
                                    None if ys is None else dw.data_ptr(),
                                    _stream_of(stream, dev, dout, ys, row_of_slot, weights))
    if st:
        _check(st, "gsa_moe_unpermute_bwd")
    return dys if want_dys else None, dw if ys is not None else None


# ---------------------------------------- grouped products of quantized operands

def _operand(q: dict, side: str, recipe_kind: int, experts: int, what: str, dev):
    """QIn of one copy of a quantized tensor (side 'row' or 'col'), and its tensors."""
    u8 = _torch.uint8
    data, scale, amax = q.get(side + "_data"), q.get(side + "_scale"), None
    if data is None or scale is None:
        raise GsaError(1, f"{what}: no {side}_data or {side}_scale (a {side} copy with tiled scales is needed)")
    if getattr(scale, "scale_layout", SCALES_TILED) != SCALES_TILED:
        raise GsaError(1, f"{what}: compact scales (a copy written with scale_layout=SCALES_TILED is needed)")
    for t in (data, scale):
        if t.dtype is not u8 or not t.is_contiguous() or t.device != dev:
            raise GsaError(1, f"{what}: contiguous uint8 {side} copy on {dev} expected")
    pa = None
    if recipe_kind == NVFP4:
        amax = q.get("amax_" + side)
        if amax is None or amax.dtype is not _torch.float32 or not amax.is_contiguous() or amax.device != dev or \
                amax.numel() < experts:
            raise GsaError(1, f"{what}: contiguous float32 amax_{side} of {experts} experts on {dev} expected")
        pa = amax.data_ptr()
    return QIn(data.data_ptr(), scale.data_ptr(), pa, data.numel(), scale.numel()), data, scale, amax


def _product_args(what, split, out_dtype):
    torch = _torch or _setup()
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise GsaError(1, f"{what}: output type {out_dtype} (bfloat16 or float32 expected)")
    if split.dim() != 1:
        raise GsaError(1, f"{what}: split must be [experts]")
    _require(split, what + ": split", split.shape, torch.int64)
    return split.device, split.shape[0], BF16 if out_dtype is torch.bfloat16 else FP32


def grouped_gemm(a: dict, b: dict, split, m: int, n: int, k: int, recipe_kind: int, out_dtype=None,
                 b_columnwise: bool = False, out=None, stream=None):
    """out [m, n] = A B_e^T over the rows of each expert, on the quantized copies that fwd / bwd write with
    scale_layout=SCALES_TILED (their compact scales are refused, buffers of the caller's own are taken as tiled).
    a: the rowwise copy of the [m, k] rows.  b: the experts' weights, the rowwise copy of [E * n, k] split into E
    times n rows, or with b_columnwise the columnwise copy of [E * k, n] split into E times k rows (the input
    gradient's product with weights [k, n]).  split: [E] int64 on the device, sum at most m (rows past it become
    zero).  out_dtype: torch.bfloat16 (default) or torch.float32."""
    torch = _torch or _setup()
    out_dtype = out_dtype or (out.dtype if out is not None else torch.bfloat16)
    dev, experts, code = _product_args("grouped_gemm", split, out_dtype)
    qa, *ta = _operand(a, "row", recipe_kind, experts, "grouped_gemm: a", dev)
    qb, *tb = _operand(b, "col" if b_columnwise else "row", recipe_kind, experts, "grouped_gemm: b", dev)
    out = _out(out, "grouped_gemm: out", (m, n), out_dtype, dev, stream)
    st = _lib.gsa_grouped_gemm(qa, qb, split.data_ptr(), experts, m, n, k, recipe_kind, out.data_ptr(), code,
                               _stream_of(stream, dev, split, *ta, *tb))
    if st:
        _check(st, "gsa_grouped_gemm")
    return out


def grouped_gemm_wgrad(a: dict, b: dict, split, m: int, n: int, k: int, recipe_kind: int, out_dtype=None,
                       out=None, accumulate: bool = False, stream=None):
    """dw [experts, n, k]: for each expert the product A^T B over its rows, from the columnwise copies (tiled scales)
    of the [m, n] and [m, k] tensors.  out_dtype: torch.float32 (default) or torch.bfloat16.  accumulate adds to
    `out`.  NVFP4 copies made with the RHT need the same sign mask on both sides."""
    torch = _torch or _setup()
    out_dtype = out_dtype or (out.dtype if out is not None else torch.float32)
    dev, experts, code = _product_args("grouped_gemm_wgrad", split, out_dtype)
    if accumulate and out is None:
        raise GsaError(1, "grouped_gemm_wgrad: accumulate needs out")
    qa, *ta = _operand(a, "col", recipe_kind, experts, "grouped_gemm_wgrad: a", dev)
    qb, *tb = _operand(b, "col", recipe_kind, experts, "grouped_gemm_wgrad: b", dev)
    out = _out(out, "grouped_gemm_wgrad: out", (experts, n, k), out_dtype, dev, stream)
    nbytes = _lib.gsa_grouped_gemm_wgrad_workspace_size(experts, m, n, k, recipe_kind)
    ws = _out(None, "", (max(256, nbytes),), torch.uint8, dev, stream)
    st = _lib.gsa_grouped_gemm_wgrad(qa, qb, split.data_ptr(), experts, m, n, k, recipe_kind, out.data_ptr(), code,
                                     1 if accumulate else 0, ws.data_ptr(), nbytes,
                                     _stream_of(stream, dev, split, *ta, *tb))
    if st:
        _check(st, "gsa_grouped_gemm_wgrad")
    return out


def _activation(what, act, params, b_groups):
    """(activation code, its parameters) of a gated projection."""
    kind = ACT.get(act) if isinstance(act, str) else int(act)
    if kind not in GLU_ACTS:
        raise GsaError(1, f"{what}: activation {act} (swiglu or clamped_swiglu expected)")
    if b_groups != 1 and b_groups != 2:
        raise GsaError(1, f"{what}: b_groups {b_groups} (1 or 2 expected)")
    return kind, params or act_params(kind)


def _gated(what, act, params, probs, m, b_groups, dev):
    """The same, and the pointer of probs [m] or None."""
    kind, prm = _activation(what, act, params, b_groups)
    if probs is None:
        return kind, prm, None
    _require(probs, what, (m,), _torch.float32)
    _same_device(what, dev, probs)
    return kind, prm, probs.data_ptr()


def grouped_glu(a: dict, b: dict, split, m: int, n: int, k: int, recipe_kind: int, act="swiglu", probs=None,
                params: ActParams | None = None, b_groups: int = 1, out_dtype=None, out=None, stream=None):
    """The gated first projection in one product: y [m, n] = probs * act(A Bg_e^T, A Bl_e^T) over the rows of each expert,
    act "swiglu" or "clamped_swiglu", probs [m] FP32 (None: 1).  a, split as for grouped_gemm.  b: the rowwise copy of the
    experts' weights [E * 2 n, k], n gate rows and then n linear rows an expert, quantized in E groups of 2 n rows
    (b_groups 1, n a multiple of 128) or 2 E groups of n rows (b_groups 2; fwd takes 256 groups, but a copy made in E groups
    becomes one of 2 E with its scale tiles laid out anew and each amax twice, as in examples/moe_ffn.py).  out_dtype:
    torch.bfloat16 (default) or torch.float32.  The pre-activations stay in FP32 and are not written: grouped_glu_bwd multiplies again."""
    torch = _torch or _setup()
    out_dtype = out_dtype or (out.dtype if out is not None else torch.bfloat16)
    dev, experts, code = _product_args("grouped_glu", split, out_dtype)
    kind, prm, pp = _gated("grouped_glu", act, params, probs, m, b_groups, dev)
    qa, *ta = _operand(a, "row", recipe_kind, experts, "grouped_glu: a", dev)
    qb, *tb = _operand(b, "row", recipe_kind, experts * b_groups, "grouped_glu: b", dev)
    out = _out(out, "grouped_glu: out", (m, n), out_dtype, dev, stream)
    st = _lib.gsa_grouped_glu(qa, qb, split.data_ptr(), experts, m, n, k, recipe_kind, kind, prm, pp, b_groups,
                              out.data_ptr(), code, _stream_of(stream, dev, split, probs, *ta, *tb))
    if st:
        _check(st, "gsa_grouped_glu")
    return out


def grouped_glu_bwd(dy, a: dict, b: dict, split, m: int, n: int, k: int, recipe_kind: int, act="swiglu", probs=None,
                    params: ActParams | None = None, b_groups: int = 1, want_dx: bool = True, want_dprobs: bool = True,
                    out_dtype=None, out: tuple | None = None, stream=None):
    """Gradient of grouped_glu for dy [m, n] BF16: (dx [m, 2 n], the pre-activations' gradient, dprobs [m] FP32), None in
    the place of what is not wanted.  The other arguments are the forward's; the rows' and the weights' gradients are
    grouped_gemm and grouped_gemm_wgrad of quantized dx."""
    torch = _torch or _setup()
    dx, dprobs = out if out is not None else (None, None)
    out_dtype = out_dtype or (dx.dtype if dx is not None else torch.bfloat16)
    dev, experts, code = _product_args("grouped_glu_bwd", split, out_dtype)
    kind, prm, pp = _gated("grouped_glu_bwd", act, params, probs, m, b_groups, dev)
    _require(dy, "grouped_glu_bwd: dy", (m, n), torch.bfloat16)
    _same_device("grouped_glu_bwd", dev, dy)
    qa, *ta = _operand(a, "row", recipe_kind, experts, "grouped_glu_bwd: a", dev)
    qb, *tb = _operand(b, "row", recipe_kind, experts * b_groups, "grouped_glu_bwd: b", dev)
    dx = _out(dx, "grouped_glu_bwd: dx", (m, 2 * n), out_dtype, dev, stream) if want_dx else None
    ws, nbytes = None, 0
    if want_dprobs:
        dprobs = _out(dprobs, "grouped_glu_bwd: dprobs", (m,), torch.float32, dev, stream)
        nbytes = _lib.gsa_grouped_glu_bwd_workspace_size(m, n)
        ws = _out(None, "", (max(256, nbytes),), torch.uint8, dev, stream)
    st = _lib.gsa_grouped_glu_bwd(dy.data_ptr(), qa, qb, split.data_ptr(), experts, m, n, k, recipe_kind, kind, prm, pp, b_groups,
                                  dx.data_ptr() if want_dx else None, code, dprobs.data_ptr() if want_dprobs else None,
                                  ws.data_ptr() if want_dprobs else None, nbytes,
                                  _stream_of(stream, dev, dy, split, probs, *ta, *tb))
    if st:
        _check(st, "gsa_grouped_glu_bwd")
    return dx, dprobs if want_dprobs else None


_few_bytes: dict = {}   # workspace bytes by sizes


def _few_rows(what, x, b, split, b_groups, recipe_kind, n, out_dtype, out, stream, act=None):
    """A product of unquantized rows.  act: (activation code, parameters, probs) of a gated one."""
    dt, dev = x.dtype, x.device
    x_code = _DTYPES.get(dt)
    if x_code is None or x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise GsaError(1, f"{what}: x must be contiguous CUDA bfloat16, float16 or float32 [rows, k], got {x.device} {dt} "
                          f"{list(x.shape)}{'' if x.is_contiguous() else ' (not contiguous)'}")
    m, k = x.shape
    sp, experts = None, 1
    if split is not None:
        if split.dtype is not _torch.int64 or split.dim() != 1 or not split.is_cuda or not split.is_contiguous():
            raise GsaError(1, f"{what}: contiguous CUDA int64 [experts] split expected, got {split.device} {split.dtype} {list(split.shape)}")
        if split.device != dev:
            _same_device(what, dev, split)
        sp, experts = split.data_ptr(), split.numel()
    kind = prm = probs = pp = None
    if act is not None:
        kind, prm, probs = act
        if probs is not None:
            _require(probs, what, (m,), _torch.float32)
            _same_device(what, dev, probs)
            pp = probs.data_ptr()
    qb, data, scale, amax = _operand(b, "row", recipe_kind, experts * b_groups, what, dev)
    if out_dtype is None:
        out_dtype, code = (dt, x_code) if out is None else (out.dtype, _DTYPES.get(out.dtype))
    else:
        code = _DTYPES.get(out_dtype)
    if code is None:
        raise GsaError(1, f"{what}: output type {out_dtype} (bfloat16, float16 or float32 expected)")
    key = (experts, m, k, recipe_kind)
    nbytes = _few_bytes.get(key)
    if nbytes is None:
        if len(_few_bytes) > 4096:
            _few_bytes.clear()
        nbytes = _few_bytes[key] = _lib.gsa_grouped_gemv_workspace_size(*key)
    out = _out(out, what, (m, n), out_dtype, dev, stream)
    ws = _out(None, "", (nbytes or 256,), _torch.uint8, dev, stream)
    s = _stream_of(stream, dev, x, split, probs, data, scale, amax)
    if act is None:
        st = _lib.gsa_grouped_gemv(x.data_ptr(), x_code, qb, sp, experts, m, n, k, recipe_kind, out.data_ptr(), code, ws.data_ptr(), nbytes, s)
    else:
        st = _lib.gsa_grouped_glu_gemv(x.data_ptr(), x_code, qb, sp, experts, m, n, k, recipe_kind, kind, prm, pp, b_groups,
                                       out.data_ptr(), code, ws.data_ptr(), nbytes, s)
    if st:
        _check(st, "gsa_" + what)
    return out


def grouped_gemv(x, b: dict, split, n: int, recipe_kind: int, out_dtype=None, out=None, stream=None):
    """out [rows, n] = x B_e^T over the rows of each expert, for a few unquantized rows an expert (decoding): x [rows, k]
    bfloat16, float16 or float32; b, split as for grouped_gemm (split None: one matrix takes all rows).  out_dtype: any
    of the three (default: x's).  x keeps its precision: values within 2^-22 of the largest one of their block of 16 (NVFP4)
    or 32 (MXFP8); blocks whose largest value is less than 2^-16 (NVFP4; MXFP8 2^-80) of the row's within 2^-37 of the row's.
    A row with a NaN or with more than eight infinite values gives NaN."""
    _torch or _setup()
    return _few_rows("grouped_gemv", x, b, split, 1, recipe_kind, n, out_dtype, out, stream)


def grouped_glu_gemv(x, b: dict, split, n: int, recipe_kind: int, act="swiglu", probs=None, params: ActParams | None = None,
                     b_groups: int = 1, out_dtype=None, out=None, stream=None):
    """grouped_glu for a few unquantized rows an expert: y [rows, n] = probs * act(x Bg_e^T, x Bl_e^T), x as for
    grouped_gemv, the rest as for grouped_glu."""
    _torch or _setup()
    kind, prm = _activation("grouped_glu_gemv", act, params, b_groups)
    return _few_rows("grouped_glu_gemv", x, b, split, b_groups, recipe_kind, n, out_dtype, out, stream, (kind, prm, probs))


def grouped_gemm_status(stream=None) -> int:
    """Takes one report of the grouped products on the current device (synchronizes the stream): 6 (a bounded wait ran
    out), 1 (a bad device split: that call wrote nothing, an output it allocated holds anything) or 0."""
    return load().gsa_grouped_gemm_status(_stream_ptr(stream))
