"""ctypes binding of libmoe's block operators (include/moe_block.h): argument
checks and marshalling only, as in _lib.

Tensors are torch tensors of their own types (bfloat16, float16, float32, int32)
on one GPU. A call runs on that GPU's current stream unless `stream` gives
another; outputs and workspaces are the caller's.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext

from . import _lib
from ._lib import _check

EXPORTS = ("moe_grouped_mm", "moe_grouped_mm_backward_workspace", "moe_grouped_mm_backward",
           "moe_linear", "moe_linear_backward_workspace", "moe_linear_backward",
           "moe_block_norm", "moe_block_norm_backward_workspace", "moe_block_norm_backward",
           "moe_combine_backward")

BF16, FP16, F32 = 0, 1, 2
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 4}
GATES = {"none": 0, "channel": 1, "token": 2, "element": 3}


class MoeMMShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "K", "N", "E", "x_rows", "topk", "dtype",
                                              "act")]


class MoeNormShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("T", "H", "dtype", "r_dtype", "y_dtype", "gate")] +
                [("scale", ctypes.c_float), ("eps", ctypes.c_float)])


_declared = False


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
            "moe_combine_backward": (INT, [P] * 5 + [I32] * 4 + [P, I32, P, P, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _declared = True
    return lib


def _ptr(t) -> int | None:
    """Device pointer; an empty tensor has none and stands as a non-null address
    that nothing reads, since NULL means that the operand is not asked for."""
    return None if t is None else t.data_ptr() or 16


def _type(t, name: str) -> int:
    import torch
    code = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: F32}.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} is {t.dtype}; bfloat16, float16 or float32 is needed")
    return code


def _half(t, name: str) -> int:
    code = _type(t, name)
    if code == F32:
        raise ValueError(f"{name} is float32; bfloat16 or float16 is needed")
    return code


def _want(t, name: str, shape, dtypes) -> None:
    """Shape, type and layout of one operand (None passes)."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, the call needs {tuple(shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} is {t.dtype}, the call needs one of "
                         f"{', '.join(str(d) for d in dtypes)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _act(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act = {act!r}; one of {', '.join(ACTS)} is needed")
    return ACTS[act]


def _disjoint(outs, ins) -> None:
    """Outputs must not overlap inputs or each other."""
    def span(t):
        a = t.data_ptr()
        return a, a + t.numel() * t.element_size()
    outs = [(n, t) for n, t in outs if t is not None and t.numel()]
    ins = [(n, t) for n, t in ins if t is not None and t.numel()]
    for i, (n, t) in enumerate(outs):
        a, b = span(t)
        for m, u in outs[i + 1:] + ins:
            c, d = span(u)
            if a < d and c < b:
                raise ValueError(f"{n} overlaps {m} in memory")


def _run(fn: str, tensors, stream, call) -> None:
    """Check that every tensor is on one device, make it current, and call."""
    import torch
    devs = {t.device for t in tensors if t is not None}
    if len(devs) > 1:
        raise ValueError(f"tensors on several devices: {sorted(str(d) for d in devs)}")
    dev = devs.pop()
    on_gpu = dev.type == "cuda"
    if not on_gpu and torch.cuda.is_available():
        raise ValueError(f"tensors on {dev}; a GPU is needed")
    other = on_gpu and dev.index != torch.cuda.current_device()
    with torch.cuda.device(dev) if other else nullcontext():
        if stream is None:
            stream = torch.cuda.current_stream(dev).cuda_stream if on_gpu else 0
        _check(fn, call(stream))


def _ws(ws):
    if ws is not None and not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size()


def _mm_dims(x, w, act, grouped):
    if w.dim() != (3 if grouped else 2) or x.dim() != 2:
        raise ValueError(f"x has shape {tuple(x.shape)}, w {tuple(w.shape)}")
    N, K = w.shape[-2:]
    if x.shape[1] != K:
        raise ValueError(f"x has {x.shape[1]} columns, w contracts {K}")
    return N, K, N // 2 if act == "swiglu" else N


def _gather(x, rows, sorted_slot, topk, expert_offsets, E):
    import torch
    _want(expert_offsets, "expert_offsets", (E + 1,), (torch.int32,))
    if sorted_slot is None:
        if x is not None and x.shape[0] != rows:
            raise ValueError(f"x has {x.shape[0]} rows, the call needs {rows}")
        return 0
    _want(sorted_slot, "sorted_slot", (rows,), (torch.int32,))
    return 0 if x is None else x.shape[0]


def grouped_mm(x, w, expert_offsets, y, sorted_slot=None, topk: int = 1, act: str = "none",
               z=None, stream=None) -> None:
    """y[p] = act(x[src(p)] W_e^T) for the rows p of each expert e.

    x [rows or tokens, K] and w [E, N, K] bfloat16 or float16; expert_offsets
    int32 [E + 1]; y [rows, N] (N / 2 for act="swiglu") of x's type or float32.
    sorted_slot int32 [rows] gathers row sorted_slot[p] // topk of x. z [rows, N]
    of x's type keeps the product for grouped_mm_backward. Rows outside
    [expert_offsets[0], expert_offsets[E]) stay as they were."""
    import torch
    dt, code = _half(x, "x"), _act(act)
    N, K, No = _mm_dims(x, w, act, True)
    E, rows = w.shape[0], y.shape[0]
    _want(x, "x", x.shape, (x.dtype,))
    _want(w, "w", (E, N, K), (x.dtype,))
    _want(y, "y", (rows, No), (x.dtype, torch.float32))
    _want(z, "z", (rows, N), (x.dtype,))
    x_rows = _gather(x, rows, sorted_slot, topk, expert_offsets, E)
    _disjoint((("y", y), ("z", z)), (("x", x), ("w", w), ("expert_offsets", expert_offsets),
                                     ("sorted_slot", sorted_slot)))
    s = MoeMMShape(rows, K, N, E, x_rows, topk, dt, code)
    _run("moe_grouped_mm", (x, w, expert_offsets, sorted_slot, y, z), stream,
         lambda st: _load().moe_grouped_mm(ctypes.byref(s), _ptr(x), _ptr(w), _ptr(expert_offsets),
                                           _ptr(sorted_slot), _ptr(z), _ptr(y), _type(y, "y"), st))


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
    they were. ws: grouped_mm_backward_workspace bytes."""
    import torch
    dt, code = _half(x, "x"), _act(act)
    N, K, No = _mm_dims(x, w, act, True)
    E, rows = w.shape[0], dy.shape[0]
    _want(x, "x", x.shape, (x.dtype,))
    _want(w, "w", (E, N, K), (x.dtype,))
    _want(dy, "dy", (rows, No), (x.dtype,))
    _want(z, "z", (rows, N), (x.dtype,))
    _want(dx, "dx", (rows, K), (x.dtype, torch.float32))
    _want(dw, "dw", (E, N, K), (x.dtype, torch.float32))
    x_rows = _gather(x, rows, sorted_slot, topk, expert_offsets, E)
    _disjoint((("dx", dx), ("dw", dw), ("ws", ws)),
              (("dy", dy), ("x", x), ("w", w), ("z", z), ("expert_offsets", expert_offsets),
               ("sorted_slot", sorted_slot)))
    s = MoeMMShape(rows, K, N, E, x_rows, topk, dt, code)
    wp, wn = _ws(ws)
    _run("moe_grouped_mm_backward", (dy, x, w, expert_offsets, sorted_slot, z, dx, dw, ws), stream,
         lambda st: _load().moe_grouped_mm_backward(
             ctypes.byref(s), _ptr(dy), _ptr(x), _ptr(w), _ptr(z), _ptr(expert_offsets),
             _ptr(sorted_slot), _ptr(dx), dt if dx is None else _type(dx, "dx"), _ptr(dw),
             dt if dw is None else _type(dw, "dw"), wp, wn, st))


def linear(x, w, y, bias=None, residual=None, act: str = "none", z=None, stream=None) -> None:
    """y = act(x W^T + bias) + residual: x [rows, K], w [N, K], bias [N] bfloat16
    or float16; y [rows, N] (N / 2 for act="swiglu") of x's type or float32;
    residual like y, or y itself. z [rows, N] keeps the product (with its bias)
    for linear_backward."""
    import torch
    dt, code = _half(x, "x"), _act(act)
    N, K, No = _mm_dims(x, w, act, False)
    rows = x.shape[0]
    _want(x, "x", (rows, K), (x.dtype,))
    _want(w, "w", (N, K), (x.dtype,))
    _want(bias, "bias", (N,), (x.dtype,))
    _want(y, "y", (rows, No), (x.dtype, torch.float32))
    _want(residual, "residual", (rows, No), (y.dtype,))
    _want(z, "z", (rows, N), (x.dtype,))
    in_place = residual is not None and residual.data_ptr() == y.data_ptr()
    _disjoint((("y", y), ("z", z)), (("x", x), ("w", w), ("bias", bias),
                                     ("residual", None if in_place else residual)))
    s = MoeMMShape(rows, K, N, 1, 0, 1, dt, code)
    _run("moe_linear", (x, w, bias, residual, z, y), stream,
         lambda st: _load().moe_linear(ctypes.byref(s), _ptr(x), _ptr(w), _ptr(bias),
                                       _ptr(residual), _ptr(z), _ptr(y), _type(y, "y"), st))


def linear_backward_workspace(rows: int, K: int, N: int, act: str = "none") -> int:
    """Bytes of workspace linear_backward needs."""
    s = MoeMMShape(rows, K, N, 1, 0, 1, BF16, _act(act))
    return int(_load().moe_linear_backward_workspace(ctypes.byref(s)))


def linear_backward(dy, x, w, dx=None, dw=None, dbias=None, act: str = "none", z=None, ws=None,
                    stream=None) -> None:
    """Gradients of linear: dx [rows, K], dw [N, K], dbias [N], each of x's type
    or float32 (dw and dbias alike), any of them None; dy [rows, N or N / 2] of
    x's type or float32, z the forward's (act="none": None). The residual's
    gradient is dy. ws: linear_backward_workspace bytes."""
    import torch
    dt, code = _half(x, "x"), _act(act)
    N, K, No = _mm_dims(x, w, act, False)
    rows = x.shape[0]
    _want(x, "x", (rows, K), (x.dtype,))
    _want(w, "w", (N, K), (x.dtype,))
    _want(dy, "dy", (rows, No), (x.dtype, torch.float32))
    _want(z, "z", (rows, N), (x.dtype,))
    _want(dx, "dx", (rows, K), (x.dtype, torch.float32))
    _want(dw, "dw", (N, K), (x.dtype, torch.float32))
    _want(dbias, "dbias", (N,), (x.dtype, torch.float32) if dw is None else (dw.dtype,))
    _disjoint((("dx", dx), ("dw", dw), ("dbias", dbias), ("ws", ws)),
              (("dy", dy), ("x", x), ("w", w), ("z", z)))
    s = MoeMMShape(rows, K, N, 1, 0, 1, dt, code)
    grad = dw if dw is not None else dbias
    wp, wn = _ws(ws)
    _run("moe_linear_backward", (dy, x, w, z, dx, dw, dbias, ws), stream,
         lambda st: _load().moe_linear_backward(
             ctypes.byref(s), _ptr(dy), _type(dy, "dy"), _ptr(x), _ptr(w), _ptr(z), _ptr(dx),
             dt if dx is None else _type(dx, "dx"), _ptr(dw), _ptr(dbias),
             dt if grad is None else _type(grad, "dw"), wp, wn, st))


def _norm_shape(r, y, gate, dtype, scale, eps):
    import torch
    if r.dim() != 2:
        raise ValueError(f"the residual stream has shape {tuple(r.shape)}; [T, H] is needed")
    T, H = r.shape
    kind = "none"
    if gate is not None:
        # by shape: [H] channel, [T, 1] token, [T, H] element
        kind = {(H,): "channel", (T, 1): "token", (T, H): "element"}.get(tuple(gate.shape))
        if kind is None:
            raise ValueError(f"gate has shape {tuple(gate.shape)}; ({H},), ({T}, 1) or ({T}, {H}) "
                             "is needed")
    half = {torch.bfloat16: BF16, torch.float16: FP16}.get(dtype)
    if half is None:
        raise ValueError(f"type {dtype}; bfloat16 or float16 is needed")
    rt = _type(r, "r")
    yt = half if y is None else _type(y, "y")
    return MoeNormShape(T, H, half, rt, yt, GATES[kind], scale, eps), kind


def _norm_type(r, y, *others):
    """The half type of a block norm's call: that of its weights, gate or h."""
    for t in others + (r, y):
        if t is not None and _type(t, "operand") != F32:
            return t.dtype
    import torch
    return torch.bfloat16


def block_norm(r, y=None, r_out=None, h=None, w_post=None, w_pre=None, gate=None,
               scale: float = 1.0, eps: float = 1e-6, stream=None) -> None:
    """r_out = r + scale * gate * rms_norm(y; w_post); h = rms_norm(r_out; w_pre).

    r, r_out [T, H] and y [T, H] are float32 or the half type of the rest
    (weights [H], gate, h [T, H]: bfloat16 or float16). w_post None: y is added
    as it is. y None: only h = rms_norm(r; w_pre). gate: [H], [T, 1] or [T, H]."""
    import torch
    dt = _norm_type(r, y, w_post, w_pre, gate, h)
    s, kind = _norm_shape(r, y, gate, dt, scale, eps)
    T, H = r.shape
    either = (dt, torch.float32)
    _want(r, "r", (T, H), either)
    _want(y, "y", (T, H), either)
    _want(r_out, "r_out", (T, H), (r.dtype,))
    _want(h, "h", (T, H), (dt,))
    _want(w_post, "w_post", (H,), (dt,))
    _want(w_pre, "w_pre", (H,), (dt,))
    if gate is not None:
        _want(gate, "gate", gate.shape, (dt,))
    _disjoint((("r_out", r_out), ("h", h)), (("r", r), ("y", y), ("w_post", w_post),
                                             ("w_pre", w_pre), ("gate", gate)))
    _run("moe_block_norm", (r, y, w_post, gate, w_pre, r_out, h), stream,
         lambda st: _load().moe_block_norm(ctypes.byref(s), _ptr(r), _ptr(y), _ptr(w_post),
                                           _ptr(gate), _ptr(w_pre), _ptr(r_out), _ptr(h), st))


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
    float32 for [H] and [T, 1], gate's type for [T, H]."""
    import torch
    dt = _norm_type(r_out, y, w_post, w_pre, gate, dh)
    s, kind = _norm_shape(r_out, y, gate, dt, scale, eps)
    T, H = r_out.shape
    either = (dt, torch.float32)
    _want(r_out, "r_out", (T, H), either)
    _want(dr_out, "dr_out", (T, H), (r_out.dtype,))
    _want(dh, "dh", (T, H), (dt,))
    _want(y, "y", (T, H), either)
    _want(w_post, "w_post", (H,), (dt,))
    _want(w_pre, "w_pre", (H,), (dt,))
    _want(dr, "dr", (T, H), (r_out.dtype,))
    if y is not None:
        _want(dy, "dy", (T, H), (y.dtype,))
    _want(dw_post, "dw_post", (H,), (torch.float32,))
    _want(dw_pre, "dw_pre", (H,), (torch.float32,))
    if gate is not None:
        _want(gate, "gate", gate.shape, (dt,))
        _want(dgate, "dgate", gate.shape, (dt,) if kind == "element" else (torch.float32,))
    _disjoint((("dr", dr), ("dy", dy), ("dw_post", dw_post), ("dw_pre", dw_pre),
               ("dgate", dgate), ("ws", ws)),
              (("r_out", r_out), ("dr_out", dr_out), ("dh", dh), ("y", y), ("w_post", w_post),
               ("w_pre", w_pre), ("gate", gate)))
    wp, wn = _ws(ws)
    _run("moe_block_norm_backward", (r_out, dr_out, dh, y, w_post, gate, w_pre, dr, dy, dw_post,
                                     dw_pre, dgate, ws), stream,
         lambda st: _load().moe_block_norm_backward(
             ctypes.byref(s), _ptr(r_out), _ptr(dr_out), _ptr(dh), _ptr(y), _ptr(w_post),
             _ptr(gate), _ptr(w_pre), _ptr(dr), _ptr(dy), _ptr(dw_post), _ptr(dw_pre),
             _ptr(dgate), wp, wn, st))


def combine_backward(dout, y, slot_pos, topk_w, dy=None, dtopk_w=None, topk_ids=None,
                     dlogits=None, stream=None) -> None:
    """Gradients of combine: dy [T k, H] (bfloat16, float16 or float32), dtopk_w
    float32 [T, k], and through route_topk's softmax dlogits float32 [T, E]
    (needs topk_ids); any of them None. dout float32 [T, H], y float32 [T k, H],
    slot_pos int32 with T k values, topk_w float32 [T, k]."""
    import torch
    f32, i32 = (torch.float32,), (torch.int32,)
    T, k = topk_w.shape
    H = dout.shape[1]
    _want(dout, "dout", (T, H), f32)
    _want(y, "y", (T * k, H), f32)
    _want(topk_w, "topk_w", (T, k), f32)
    if slot_pos.numel() != T * k:
        raise ValueError(f"slot_pos holds {slot_pos.numel()} values, the call needs {T * k}")
    _want(slot_pos, "slot_pos", slot_pos.shape, i32)
    _want(topk_ids, "topk_ids", (T, k), i32)
    _want(dy, "dy", (T * k, H), (torch.bfloat16, torch.float16, torch.float32))
    _want(dtopk_w, "dtopk_w", (T, k), f32)
    E = k
    if dlogits is not None:
        E = dlogits.shape[-1]
        _want(dlogits, "dlogits", (T, E), f32)
    _disjoint((("dy", dy), ("dtopk_w", dtopk_w), ("dlogits", dlogits)),
              (("dout", dout), ("y", y), ("slot_pos", slot_pos), ("topk_w", topk_w),
               ("topk_ids", topk_ids)))
    _run("moe_combine_backward", (dout, y, slot_pos, topk_w, topk_ids, dy, dtopk_w, dlogits), stream,
         lambda st: _load().moe_combine_backward(
             _ptr(dout), _ptr(y), _ptr(slot_pos), _ptr(topk_ids), _ptr(topk_w), T, H, E, k,
             _ptr(dy), F32 if dy is None else _type(dy, "dy"), _ptr(dtopk_w), _ptr(dlogits), st))
