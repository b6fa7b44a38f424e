"""Python entry points of libmoe's int8 operators (include/moe_int8.h): argument checks
and marshalling only. Tensors, streams and errors as in _block, whose binding checks the
tensors of these calls too.
"""
from __future__ import annotations

import ctypes

from . import _block, _lib
from ._block import _act, _done, _ext, _load

EXPORTS = ("moe_quant_rows", "moe_linear_w8a8_workspace", "moe_linear_w8a8",
           "moe_linear_w8a8_plan",
           "moe_layer_w8a8_workspace", "moe_layer_w8a8",
           "moe_layer_w8a8_plan")


def quant_rows(x, q, scale, stream=None) -> None:
    """int8 codes q [rows, K] and float32 scales [rows] of x [rows, K] (bfloat16,
    float16 or float32): scale = max|x| / 127, q = x / scale to the nearest whole
    number. A row with an infinity or a NaN gets the scale NaN and the codes 0."""
    args = (x, q, scale, stream)
    st = (_block._binding or _ext()).quant_rows(*args)
    if st:
        _done("moe_quant_rows", st, lambda: _block._binding.quant_rows(*args))


def linear_w8a8_workspace(rows: int, K: int) -> int:
    """Bytes of workspace linear_w8a8 needs for x that holds values, not codes."""
    return int(_load().moe_linear_w8a8_workspace(rows, K))


def linear_w8a8(x, w, w_scale, y, x_scale=None, bias=None, residual=None, act: str = "none",
                ws=None, stream=None) -> None:
    """y = act(x W^T * x_scale * w_scale + bias) + residual on int8 codes.

    w int8 [N, K] with w_scale float32 [N]. x int8 [rows, K] with x_scale float32
    [rows], or bfloat16 or float16 [rows, K]: the call then makes the codes of
    quant_rows in ws (linear_w8a8_workspace bytes). bias float32 [N]; y [rows, N]
    (N / 2 for act="swiglu") bfloat16, float16 or float32; residual like y, or y
    itself."""
    args = (x, x_scale, w, w_scale, bias, residual, y, ws, _act(act), stream)
    st = (_block._binding or _ext()).linear_w8a8(*args)
    if st:
        _done("moe_linear_w8a8", st, lambda: _block._binding.linear_w8a8(*args))


_CODES = (None, "in the launch", "before it")


def linear_w8a8_plan(rows: int, K: int, N: int, act: str = "none", codes: bool = False) -> dict:
    """The kernel that linear_w8a8 runs on for this shape, for tests and tuning: its tiles
    as product_plan names them, or "rings" of a depth; codes says where those of x are made
    (None: given)."""
    s = _block.MoeW8Shape(rows, K, N, 3 if codes else 0, 0, _act(act))
    plan = (ctypes.c_int32 * 3)()
    _lib._check("moe_linear_w8a8_plan", _load().moe_linear_w8a8_plan(ctypes.byref(s), plan))
    kernel, depth, made = plan
    return dict(kernel=(*_block._TILES, "rings")[kernel], depth=depth, codes=_CODES[made])


def layer_w8a8_workspace(T: int, H: int, I: int, E: int, k: int) -> int:
    """Bytes of workspace layer_w8a8 needs."""
    s = _lib.MoeShape(T, H, I, E, k)
    return int(_load().moe_layer_w8a8_workspace(ctypes.byref(s)))


def layer_w8a8(logits, x, w13, s13, w2, s2, topk_ids, topk_w, out, ws, residual=None,
               expert_offsets=None, stream=None) -> None:
    """The whole routed layer on int8 experts: out = residual + sum over the k picks of
    each token of topk_w * (silu(gate) up . W2^T).

    logits float32 [T, E]; x [T, H] bfloat16 or float16; w13 int8 [E, 2 I, H] (gate
    rows, then up rows) with s13 float32 [E, 2 I]; w2 int8 [E, H, I] with s2 float32
    [E, H]. Written: topk_ids int32 [T, k], topk_w float32 [T, k], out [T, H]
    (bfloat16, float16 or float32) and, where given, expert_offsets int32 [E + 1] (as
    permute's, for expert_counts_accumulate). residual like out, or out itself. ws:
    layer_w8a8_workspace bytes."""
    args = (logits, x, w13, s13, w2, s2, residual, topk_ids, topk_w, expert_offsets, out, ws,
            stream)
    st = (_block._binding or _ext()).layer_w8a8(*args)
    if st:
        _done("moe_layer_w8a8", st, lambda: _block._binding.layer_w8a8(*args))


_WAYS = ("rings", "rings by 16 rows", "tiles", "tiles of the grouped FFN")


def layer_w8a8_plan(T: int, H: int, I: int, E: int, k: int) -> dict:
    """The kernels that layer_w8a8 runs on for this shape, for tests and tuning: the way,
    and for gate_up and down (the depth of their rings or their tiles' name, where the codes
    are made)."""
    s = _lib.MoeShape(T, H, I, E, k)
    plan = (ctypes.c_int32 * 5)()
    _lib._check("moe_layer_w8a8_plan", _load().moe_layer_w8a8_plan(ctypes.byref(s), plan))
    way, up, up_codes, down, down_codes = plan
    take = (lambda v: v, lambda v: v, lambda v: _block._TILES[v], lambda v: None)[way]
    return dict(way=_WAYS[way], gate_up=(take(up), _CODES[up_codes]),
                down=(take(down), _CODES[down_codes]))
