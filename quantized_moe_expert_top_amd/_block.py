"""ctypes binding of libmoe's block operators (include/moe_block.h): argument
checks and marshalling only, as in _lib.

Tensors are torch tensors of their own types (bfloat16, float16, float32, int32)
on one GPU. A call runs on that GPU's current stream unless `stream` gives
another; outputs and workspaces are the caller's.
"""
from __future__ import annotations

import ctypes

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
    """Shape and type of one operand (None passes)."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, the call needs {tuple(shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} is {t.dtype}, the call needs one of "
                         f"{', '.join(str(d) for d in dtypes)}")


def _act(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act = {act!r}; one of {', '.join(ACTS)} is needed")
    return ACTS[act]


# Checked signatures: (entry point, scalars, shape and type of every operand) ->
# what the call passes besides pointers. Checking shapes in Python costs more than
# launching a small kernel, so it is done once per signature; whatever belongs to
# the tensors themselves (layout, device, addresses) is looked at on every call.
_plans: dict = {}
_MAX_PLANS = 4096


def _plan(key, check):
    plan = _plans.get(key)
    if plan is None:
        plan = check()
        if len(_plans) >= _MAX_PLANS:
            _plans.clear()
        _plans[key] = plan
    return plan


def _sig(tensors):
    return tuple([None if t is None else (t.shape, t.dtype) for t in tensors])


def _call(fn: str, f, names, tensors, stream, args) -> None:
    """Check layout and device of every tensor, then f(*args(pointers), stream).
    An empty tensor has no address and stands as a non-null one that nothing
    reads, since NULL means that the operand is not asked for."""
    import torch
    dev = None
    ptrs = []
    for t in tensors:
        if t is None:
            ptrs.append(None)
            continue
        if not t.is_contiguous():
            raise ValueError(f"{names[len(ptrs)]} must be contiguous")
        d = t.get_device()
        if d != dev:
            if dev is not None:
                raise ValueError(f"{names[len(ptrs)]} is on {t.device}, the operands before it "
                                 f"on {'cpu' if dev < 0 else f'cuda:{dev}'}")
            dev = d
        ptrs.append(t.data_ptr() or 16)
    if dev < 0:
        if torch.cuda.is_available():
            raise ValueError("tensors on the CPU; a GPU is needed")
        status = f(*args(ptrs), stream or 0)
    elif dev == torch._C._cuda_getDevice():
        status = f(*args(ptrs), torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream)
    else:
        with torch.cuda.device(dev):
            status = f(*args(ptrs),
                       torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream)
    if status:
        _check(fn, status)


def _bytes(ws) -> int:
    return 0 if ws is None else ws.numel() * ws.element_size()


def _mm_dims(x, w, act, grouped):
    if w.dim() != (3 if grouped else 2) or x.dim() != 2:
        raise ValueError(f"x has shape {tuple(x.shape)}, w {tuple(w.shape)}")
    N, K = w.shape[-2:]
    if x.shape[1] != K:
        raise ValueError(f"x has {x.shape[1]} columns, w contracts {K}")
    return N, K, N // 2 if act == "swiglu" else N


def _gather(x, rows, sorted_slot, expert_offsets, E):
    import torch
    _want(expert_offsets, "expert_offsets", (E + 1,), (torch.int32,))
    if sorted_slot is None:
        if x.shape[0] != rows:
            raise ValueError(f"x has {x.shape[0]} rows, the call needs {rows}")
        return 0
    _want(sorted_slot, "sorted_slot", (rows,), (torch.int32,))
    return x.shape[0]


_GROUPED = ("x", "w", "expert_offsets", "sorted_slot", "z", "y")


def grouped_mm(x, w, expert_offsets, y, sorted_slot=None, topk: int = 1, act: str = "none",
               z=None, stream=None) -> None:
    """y[p] = act(x[src(p)] W_e^T) for the rows p of each expert e.

    x [rows or tokens, K] and w [E, N, K] bfloat16 or float16; expert_offsets
    int32 [E + 1]; y [rows, N] (N / 2 for act="swiglu") of x's type or float32.
    sorted_slot int32 [rows] gathers row sorted_slot[p] // topk of x. z [rows, N]
    of x's type keeps the product for grouped_mm_backward. Rows outside
    [expert_offsets[0], expert_offsets[E]) stay as they were."""
    ts = (x, w, expert_offsets, sorted_slot, z, y)

    def check():
        import torch
        dt, code = _half(x, "x"), _act(act)
        N, K, No = _mm_dims(x, w, act, True)
        E, rows = w.shape[0], y.shape[0]
        _want(w, "w", (E, N, K), (x.dtype,))
        _want(y, "y", (rows, No), (x.dtype, torch.float32))
        _want(z, "z", (rows, N), (x.dtype,))
        x_rows = _gather(x, rows, sorted_slot, expert_offsets, E)
        return (_load().moe_grouped_mm,
                ctypes.byref(MoeMMShape(rows, K, N, E, x_rows, topk, dt, code)), _type(y, "y"))
    f, s, yt = _plan(("g", act, topk, _sig(ts)), check)
    _call("moe_grouped_mm", f, _GROUPED, ts, stream, lambda p: (s, *p, yt))


def grouped_mm_backward_workspace(rows: int, K: int, N: int, E: int, act: str = "none") -> int:
    """Bytes of workspace grouped_mm_backward needs."""
    s = MoeMMShape(rows, K, N, E, 0, 1, BF16, _act(act))
    return int(_load().moe_grouped_mm_backward_workspace(ctypes.byref(s)))


_GROUPED_BWD = ("dy", "x", "w", "z", "expert_offsets", "sorted_slot", "dx", "dw", "ws")


def grouped_mm_backward(dy, x, w, expert_offsets, dx=None, dw=None, sorted_slot=None,
                        topk: int = 1, act: str = "none", z=None, ws=None, stream=None) -> None:
    """Gradients of grouped_mm: dx [rows, K] (one row per grouped row) and
    dw [E, N, K], each of x's type or float32 and either of them None; dy
    [rows, N or N / 2] of x's type, z the forward's (act="none": None). Every
    element of dw is written; rows of dx outside the experts' blocks stay as
    they were. ws: grouped_mm_backward_workspace bytes."""
    ts = (dy, x, w, z, expert_offsets, sorted_slot, dx, dw, ws)

    def check():
        import torch
        dt, code = _half(x, "x"), _act(act)
        N, K, No = _mm_dims(x, w, act, True)
        E, rows = w.shape[0], dy.shape[0]
        _want(w, "w", (E, N, K), (x.dtype,))
        _want(dy, "dy", (rows, No), (x.dtype,))
        _want(z, "z", (rows, N), (x.dtype,))
        _want(dx, "dx", (rows, K), (x.dtype, torch.float32))
        _want(dw, "dw", (E, N, K), (x.dtype, torch.float32))
        x_rows = _gather(x, rows, sorted_slot, expert_offsets, E)
        return (_load().moe_grouped_mm_backward,
                ctypes.byref(MoeMMShape(rows, K, N, E, x_rows, topk, dt, code)),
                dt if dx is None else _type(dx, "dx"), dt if dw is None else _type(dw, "dw"))
    f, s, xt, wt = _plan(("gb", act, topk, _sig(ts[:8])), check)
    _call("moe_grouped_mm_backward", f, _GROUPED_BWD, ts, stream,
          lambda p: (s, *p[:7], xt, p[7], wt, p[8], _bytes(ws)))


_LINEAR = ("x", "w", "bias", "residual", "z", "y")


def linear(x, w, y, bias=None, residual=None, act: str = "none", z=None, stream=None) -> None:
    """y = act(x W^T + bias) + residual: x [rows, K], w [N, K], bias [N] bfloat16
    or float16; y [rows, N] (N / 2 for act="swiglu") of x's type or float32;
    residual like y, or y itself. z [rows, N] keeps the product (with its bias)
    for linear_backward."""
    ts = (x, w, bias, residual, z, y)

    def check():
        import torch
        dt, code = _half(x, "x"), _act(act)
        N, K, No = _mm_dims(x, w, act, False)
        rows = x.shape[0]
        _want(w, "w", (N, K), (x.dtype,))
        _want(bias, "bias", (N,), (x.dtype,))
        _want(y, "y", (rows, No), (x.dtype, torch.float32))
        _want(residual, "residual", (rows, No), (y.dtype,))
        _want(z, "z", (rows, N), (x.dtype,))
        return (_load().moe_linear, ctypes.byref(MoeMMShape(rows, K, N, 1, 0, 1, dt, code)),
                _type(y, "y"))
    f, s, yt = _plan(("l", act, _sig(ts)), check)
    _call("moe_linear", f, _LINEAR, ts, stream, lambda p: (s, *p, yt))


def linear_backward_workspace(rows: int, K: int, N: int, act: str = "none") -> int:
    """Bytes of workspace linear_backward needs."""
    s = MoeMMShape(rows, K, N, 1, 0, 1, BF16, _act(act))
    return int(_load().moe_linear_backward_workspace(ctypes.byref(s)))


_LINEAR_BWD = ("dy", "x", "w", "z", "dx", "dw", "dbias", "ws")


def linear_backward(dy, x, w, dx=None, dw=None, dbias=None, act: str = "none", z=None, ws=None,
                    stream=None) -> None:
    """Gradients of linear: dx [rows, K], dw [N, K], dbias [N], each of x's type
    or float32 (dw and dbias alike), any of them None; dy [rows, N or N / 2] of
    x's type or float32, z the forward's (act="none": None). The residual's
    gradient is dy. ws: linear_backward_workspace bytes."""
    ts = (dy, x, w, z, dx, dw, dbias, ws)

    def check():
        import torch
        dt, code = _half(x, "x"), _act(act)
        N, K, No = _mm_dims(x, w, act, False)
        rows = x.shape[0]
        _want(w, "w", (N, K), (x.dtype,))
        _want(dy, "dy", (rows, No), (x.dtype, torch.float32))
        _want(z, "z", (rows, N), (x.dtype,))
        _want(dx, "dx", (rows, K), (x.dtype, torch.float32))
        _want(dw, "dw", (N, K), (x.dtype, torch.float32))
        _want(dbias, "dbias", (N,), (x.dtype, torch.float32) if dw is None else (dw.dtype,))
        grad = dw if dw is not None else dbias
        return (_load().moe_linear_backward,
                ctypes.byref(MoeMMShape(rows, K, N, 1, 0, 1, dt, code)), _type(dy, "dy"),
                dt if dx is None else _type(dx, "dx"), dt if grad is None else _type(grad, "dw"))
    f, s, yt, xt, wt = _plan(("lb", act, _sig(ts[:7])), check)
    _call("moe_linear_backward", f, _LINEAR_BWD, ts, stream,
          lambda p: (s, p[0], yt, p[1], p[2], p[3], p[4], xt, p[5], p[6], wt, p[7], _bytes(ws)))


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


_NORM = ("r", "y", "w_post", "gate", "w_pre", "r_out", "h")


def block_norm(r, y=None, r_out=None, h=None, w_post=None, w_pre=None, gate=None,
               scale: float = 1.0, eps: float = 1e-6, stream=None) -> None:
    """r_out = r + scale * gate * rms_norm(y; w_post); h = rms_norm(r_out; w_pre).

    r, r_out [T, H] and y [T, H] are float32 or the half type of the rest
    (weights [H], gate, h [T, H]: bfloat16 or float16). w_post None: y is added
    as it is. y None: only h = rms_norm(r; w_pre). gate: [H], [T, 1] or [T, H]."""
    ts = (r, y, w_post, gate, w_pre, r_out, h)

    def check():
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
        return _load().moe_block_norm, ctypes.byref(s)
    f, s = _plan(("n", scale, eps, _sig(ts)), check)
    _call("moe_block_norm", f, _NORM, ts, stream, lambda p: (s, *p))


def block_norm_backward_workspace(T: int, H: int) -> int:
    """Bytes of workspace block_norm_backward needs for gradients of weights and
    of a channel gate."""
    return int(_load().moe_block_norm_backward_workspace(T, H))


_NORM_BWD = ("r_out", "dr_out", "dh", "y", "w_post", "gate", "w_pre", "dr", "dy", "dw_post",
             "dw_pre", "dgate", "ws")


def block_norm_backward(r_out, dr, dh=None, dr_out=None, y=None, w_post=None, w_pre=None,
                        gate=None, scale: float = 1.0, eps: float = 1e-6, dy=None, dw_post=None,
                        dw_pre=None, dgate=None, ws=None, stream=None) -> None:
    """Gradients of block_norm from dr_out [T, H] (r_out's type) and dh [T, H],
    either of them None. r_out is the forward's (r itself where y was None). dr
    like r_out; dy like y; dw_post, dw_pre float32 [H]; dgate shaped like gate,
    float32 for [H] and [T, 1], gate's type for [T, H]."""
    ts = (r_out, dr_out, dh, y, w_post, gate, w_pre, dr, dy, dw_post, dw_pre, dgate, ws)

    def check():
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
        return _load().moe_block_norm_backward, ctypes.byref(s)
    f, s = _plan(("nb", scale, eps, _sig(ts[:12])), check)
    _call("moe_block_norm_backward", f, _NORM_BWD, ts, stream, lambda p: (s, *p, _bytes(ws)))


_COMBINE_BWD = ("dout", "y", "slot_pos", "topk_ids", "topk_w", "dy", "dtopk_w", "dlogits")


def combine_backward(dout, y, slot_pos, topk_w, dy=None, dtopk_w=None, topk_ids=None,
                     dlogits=None, stream=None) -> None:
    """Gradients of combine: dy [T k, H] (bfloat16, float16 or float32), dtopk_w
    float32 [T, k], and through route_topk's softmax dlogits float32 [T, E]
    (needs topk_ids); any of them None. dout float32 [T, H], y float32 [T k, H],
    slot_pos int32 with T k values, topk_w float32 [T, k]."""
    ts = (dout, y, slot_pos, topk_ids, topk_w, dy, dtopk_w, dlogits)

    def check():
        import torch
        f32, i32 = (torch.float32,), (torch.int32,)
        if topk_w.dim() != 2 or dout.dim() != 2:
            raise ValueError(f"topk_w has shape {tuple(topk_w.shape)}, dout {tuple(dout.shape)}")
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
        return _load().moe_combine_backward, T, H, E, k, F32 if dy is None else _type(dy, "dy")
    f, T, H, E, k, yt = _plan(("cb", _sig(ts)), check)
    _call("moe_combine_backward", f, _COMBINE_BWD, ts, stream,
          lambda p: (p[0], p[1], p[2], p[3], p[4], T, H, E, k, p[5], yt, p[6], p[7]))
