"""The largest products of the block operators: what is refused, before anything is
enqueued, and what is not (host only: no kernels run here)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

try:
    from quantized_moe_expert_top_amd import _block
    LIB = _block._load()
except RuntimeError:  # not built
    LIB = None

pytestmark = pytest.mark.skipif(LIB is None, reason="libmoe.so not built")

NO_GPU = not torch.cuda.is_available()
ESHAPE, EDEV = 2, 6
BF, F32 = 0, 2
FAR = [(i + 1) << 42 for i in range(16)]     # places for operands, never dereferenced


def shape(rows, K, N, E=1, act=0):
    return ctypes.byref(_block.MoeMMShape(rows, K, N, E, rows, 1, BF, act))


def forward(s, grouped):
    x, w, off, z, y = FAR[:5]
    if grouped:
        return LIB.moe_grouped_mm(s, x, w, off, None, z, y, BF, None)
    return LIB.moe_linear(s, x, w, None, None, z, y, BF, None)


def backward(s, grouped, dx=True, dw=True):
    dy, x, w, z, off, pdx, pdw, ws = FAR[:8]
    pdx, pdw = pdx if dx else None, pdw if dw else None
    n = 1 << 41
    if grouped:
        return LIB.moe_grouped_mm_backward(s, dy, x, w, z, off, None, pdx, BF, pdw, BF, ws, n, None)
    return LIB.moe_linear_backward(s, dy, BF, x, w, z, pdx, BF, pdw, FAR[8], BF, ws, n, None)


@pytest.mark.parametrize("act", [0, 4])
def test_a_gradient_whose_launch_is_too_large_is_refused_first(act):
    """Weight gradients of 2^40 values: 2^24 tiles of 256x256 with 512 threads each. The
    call is refused as a whole, before the activation's gradient or dx is launched."""
    s = shape(4, 1 << 15, 1 << 15, E=1024, act=act)
    for dx in (True, False):
        assert backward(s, True, dx=dx) == ESHAPE
        assert b"2^32 threads" in LIB.moe_last_error()
    if NO_GPU:
        assert backward(s, True, dw=False) == EDEV and forward(s, True) == EDEV
