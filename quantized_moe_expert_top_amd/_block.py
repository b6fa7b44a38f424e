"""Python entry points of libmoe's block operators (include/moe_block.h): argument
checks and marshalling only, as in _lib. The checks of a call's tensors are made in
csrc/block_binding.cpp.

Tensors are torch tensors of their own types (bfloat16, float16, float32, int32),
contiguous, on one GPU. A call runs on that GPU's current stream unless `stream`
gives another; outputs and workspaces are the caller's. ValueError: a tensor whose
shape, type, layout or device does not fit the call; MoeError: what the library
refuses.
"""
from __future__ import annotations

import ctypes
import os

from . import _lib
from ._lib import _check

EXPORTS = ("moe_grouped_mm", "moe_grouped_mm_backward_workspace", "moe_grouped_mm_backward",
           "moe_linear", "moe_linear_backward_workspace", "moe_linear_backward",
           "moe_block_norm", "moe_block_norm_backward_workspace", "moe_block_norm_backward",
           "moe_combine_backward", "moe_product_plan")

BF16, FP16, F32 = 0, 1, 2
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 4}


class MoeMMShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "K", "N", "E", "x_rows", "topk", "dtype",
                                              "act")]


class MoeNormShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("T", "H", "dtype", "r_dtype", "y_dtype", "gate")] +
                [("scale", ctypes.c_float), ("eps", ctypes.c_float)])


BINDING_PATH = os.path.join(_lib.HERE, "_block_binding.so")
_CALLS = ("moe_grouped_mm", "moe_grouped_mm_backward", "moe_linear", "moe_linear_backward",
          "moe_block_norm", "moe_block_norm_backward", "moe_combine_backward")

_declared = False
_binding = None


def _load() -> ctypes.CDLL:
    global _declared
    lib = _lib.load()
    if not _declared:
        P, I32, SZ, INT = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int
        mm, norm = ctypes.POINTER(MoeMMShape), ctypes.POINTER(MoeNormShape)
        sig = {
            "moe_grouped_mm": (INT, [mm] + [P] * 6 + [I32, P]),
            "moe_grouped_mm_backward_workspace": (SZ, [mm]),
            "moe_grouped_mm_backward": (INT, [mm] + [P] * 7 + [I32, P, I32, P, SZ, P]),
            "moe_linear": (INT, [mm] + [P] * 6 + [I32, P]),
            "moe_linear_backward_workspace": (SZ, [mm]),
            "moe_linear_backward": (INT, [mm, P, I32, P, P, P, P, I32, P, P, I32, P, SZ, P]),
            "moe_block_norm": (INT, [norm] + [P] * 8),
            "moe_block_norm_backward_workspace": (SZ, [I32, I32]),
            "moe_block_norm_backward": (INT, [norm] + [P] * 13 + [SZ, P]),
            "moe_product_plan": (INT, [mm, I32, P]),
            "moe_combine_backward": (INT, [P] * 5 + [I32] * 4 + [P, I32, P, P, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _declared = True
    return lib


def _ext():
    """The binding module, loaded once and given libmoe's entry points."""
    global _binding
    if _binding is None:
        lib = _load()
        import importlib.machinery
        import importlib.util
        import torch
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"the binding is not built at {BINDING_PATH}; run "
                               "__graft_entry__.build() or "
                               "python -m quantized_moe_expert_top_amd.build")
        loader = importlib.machinery.ExtensionFileLoader("_block_binding", BINDING_PATH)
        spec = importlib.util.spec_from_file_location("_block_binding", BINDING_PATH, loader=loader)
        mod = importlib.util.module_from_spec(spec)
        loader.exec_module(mod)
        gpu = torch.cuda.is_available()
        if gpu:
            torch.cuda.init()
        mod.init(*[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _CALLS],
                 getattr(torch._C, "_cuda_getDevice", None),
                 getattr(torch._C, "_cuda_getCurrentRawStream", None), gpu)
        _binding = mod
    return _binding


def _done(fn: str, status: int, call) -> None:
    """Raise on a status; below zero, repeat `call` with GPU -1 - status current."""
    if status < 0:
        import torch
        with torch.cuda.device(-1 - status):
            status = call()
    if status:
        _check(fn, status)


def _act(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act = {act!r}; one of {', '.join(ACTS)} is needed")
    return ACTS[act]


def grouped_mm(x, w, expert_offsets, y, sorted_slot=None, topk: int = 1, act: str = "none",
               z=None, stream=None) -> None:
    """y[p] = act(x[src(p)] W_e^T) for the rows p of each expert e.

    x [rows or tokens, K] and w [E, N, K] bfloat16 or float16; expert_offsets
    int32 [E + 1]; y [rows, N] (N / 2 for act="swiglu") of x's type or float32.
    sorted_slot int32 [rows] gathers row sorted_slot[p] // topk of x. z [rows, N]
    of x's type keeps the product for grouped_mm_backward. Rows outside
    [expert_offsets[0], expert_offsets[E]) stay as they were."""
    args = (x, w, expert_offsets, sorted_slot, z, y, topk, _act(act), stream)
    st = (_binding or _ext()).grouped_mm(*args)
    if st:
        _done("moe_grouped_mm", st, lambda: _binding.grouped_mm(*args))


def grouped_mm_backward_workspace(rows: int, K: int, N: int, E: int, act: str = "none") -> int:
    """Bytes of workspace grouped_mm_backward needs."""
    s = MoeMMShape(rows, K, N, E, 0, 1, BF16, _act(act))
    return int(_load().moe_grouped_mm_backward_workspace(ctypes.byref(s)))


def grouped_mm_backward(dy, x, w, expert_offsets, dx=None, dw=None, sorted_slot=None,
                        topk: int = 1, act: str = "none", z=None, ws=None, stream=None) -> None:
    """Gradients of grouped_mm: dx [rows, K] (one row per grouped row) and
    dw [E, N, K], each of x's type or float32 and either of them None; dy
    [rows, N or N / 2] of x's type, z the forward's (act="none": None). Every
    element of dw is written; rows of dx outside the experts' blocks stay as
    they were. act'(z) dy enters the products in x's type: for float16 under 2^-25 it
    is zero, from 65520 on infinite. ws: grouped_mm_backward_workspace bytes."""
    args = (dy, x, w, z, expert_offsets, sorted_slot, dx, dw, ws, topk, _act(act), stream)
    st = (_binding or _ext()).grouped_mm_backward(*args)
    if st:
        _done("moe_grouped_mm_backward", st, lambda: _binding.grouped_mm_backward(*args))


def linear(x, w, y, bias=None, residual=None, act: str = "none", z=None, stream=None) -> None:
    """y = act(x W^T + bias) + residual: x [rows, K], w [N, K], bias [N] bfloat16
    or float16; y [rows, N] (N / 2 for act="swiglu") of x's type or float32;
    residual like y, or y itself. z [rows, N] keeps the product (with its bias)
    for linear_backward."""
    args = (x, w, bias, residual, z, y, _act(act), stream)
    st = (_binding or _ext()).linear(*args)
    if st:
        _done("moe_linear", st, lambda: _binding.linear(*args))


def linear_backward_workspace(rows: int, K: int, N: int, act: str = "none") -> int:
    """Bytes of workspace linear_backward needs."""
    s = MoeMMShape(rows, K, N, 1, 0, 1, BF16, _act(act))
    return int(_load().moe_linear_backward_workspace(ctypes.byref(s)))


def linear_backward(dy, x, w, dx=None, dw=None, dbias=None, act: str = "none", z=None, ws=None,
                    stream=None) -> None:
    """Gradients of linear: dx [rows, K], dw [N, K], dbias [N], each of x's type
    or float32 (dw and dbias alike), any of them None; dy [rows, N or N / 2] of
    x's type or float32, z the forward's (act="none": None). The residual's
    gradient is dy. act'(z) dy enters dx and dw in x's type, float32 dy or not: for
    float16 under 2^-25 it is zero, from 65520 on infinite. ws:
    linear_backward_workspace bytes."""
    args = (dy, x, w, z, dx, dw, dbias, ws, _act(act), stream)
    st = (_binding or _ext()).linear_backward(*args)
    if st:
        _done("moe_linear_backward", st, lambda: _binding.linear_backward(*args))


_TILES = ("256x256", "128x128", "64x128", "64x64", "128x256", "128x128 deep", "rows by 16",
          "rows by 32")
_DW_TILES = ("256x256", "256x128", "128x128", "64x64")


def product_plan(rows: int, K: int, N: int, E: int = 0, act: str = "none") -> dict:
    """The kernels that linear (E = 0) or grouped_mm and their gradients run on for
    this shape, for tests and tuning: forward, dx and dw name tiles, dx_parts and
    dw_parts count the parts of their contractions, together names the tiles of the
    one launch for both gradients (None: each in its own)."""
    s = MoeMMShape(rows, K, N, E or 1, 0, 1, BF16, _act(act))
    plan = (ctypes.c_int32 * 6)()
    _check("moe_product_plan", _load().moe_product_plan(ctypes.byref(s), E > 0, plan))
    f, pair, dx, dx_parts, dw, dw_parts = plan
    return dict(forward=_TILES[f], together=(None, "128x128", "64x64")[pair], dx=_TILES[dx],
                dx_parts=dx_parts, dw=_DW_TILES[dw], dw_parts=dw_parts)


def block_norm(r, y=None, r_out=None, h=None, w_post=None, w_pre=None, gate=None,
               scale: float = 1.0, eps: float = 1e-6, stream=None) -> None:
    """r_out = r + scale * gate * rms_norm(y; w_post); h = rms_norm(r_out; w_pre).

    r, r_out [T, H] and y [T, H] are float32 or the half type of the rest
    (weights [H], gate, h [T, H]: bfloat16 or float16). w_post None: y is added
    as it is. y None: only h = rms_norm(r; w_pre). gate: [H], [T, 1] or [T, H]."""
    args = (r, y, w_post, gate, w_pre, r_out, h, scale, eps, stream)
    st = (_binding or _ext()).block_norm(*args)
    if st:
        _done("moe_block_norm", st, lambda: _binding.block_norm(*args))


def block_norm_backward_workspace(T: int, H: int) -> int:
    """Bytes of workspace block_norm_backward needs for gradients of weights and
    of a channel gate."""
    return int(_load().moe_block_norm_backward_workspace(T, H))


def block_norm_backward(r_out, dr, dh=None, dr_out=None, y=None, w_post=None, w_pre=None,
                        gate=None, scale: float = 1.0, eps: float = 1e-6, dy=None, dw_post=None,
                        dw_pre=None, dgate=None, ws=None, stream=None) -> None:
    """Gradients of block_norm from dr_out [T, H] (r_out's type) and dh [T, H],
    either of them None. r_out is the forward's (r itself where y was None). dr
    like r_out; dy like y; dw_post, dw_pre float32 [H]; dgate shaped like gate,
    float32 for [H] and [T, 1], gate's type for [T, H]. ws:
    block_norm_backward_workspace bytes, where dw_post, dw_pre or a channel gate's
    gradient is asked for."""
    args = (r_out, dr_out, dh, y, w_post, gate, w_pre, dr, dy, dw_post, dw_pre, dgate, ws, scale,
            eps, stream)
    st = (_binding or _ext()).block_norm_backward(*args)
    if st:
        _done("moe_block_norm_backward", st, lambda: _binding.block_norm_backward(*args))


def combine_backward(dout, y, slot_pos, topk_w, dy=None, dtopk_w=None, topk_ids=None,
                     dlogits=None, stream=None) -> None:
    """Gradients of combine: dy [T k, H] (bfloat16, float16 or float32), dtopk_w
    float32 [T, k], and through route_topk's softmax dlogits float32 [T, E]
    (needs topk_ids); any of them None. dout float32 [T, H], y float32 [T k, H],
    slot_pos int32 with T k values, topk_w float32 [T, k]."""
    args = (dout, y, slot_pos, topk_ids, topk_w, dy, dtopk_w, dlogits, stream)
    st = (_binding or _ext()).combine_backward(*args)
    if st:
        _done("moe_combine_backward", st, lambda: _binding.combine_backward(*args))
