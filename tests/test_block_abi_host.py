"""Host-only checks of the block operators' C ABI and binding: exports, every
refusal before any device work, workspace sizes (no kernels run here)."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_block.h")

try:
    from quantized_moe_expert_top_amd import _block, _lib
    LIB = _block._load()
except RuntimeError as exc:  # not built
    LIB = None
    REASON = str(exc)

pytestmark = pytest.mark.skipif(LIB is None, reason="libmoe.so not built")

A = 0x10000          # a 16-byte aligned stand-in address, never dereferenced on the host
MIS = 0x10008        # misaligned


def place(*args):
    """A place of its own for every operand that stands at A (2^32 bytes apart)."""
    return [(i + 1) << 32 if v == A else v for i, v in enumerate(args)]


BIG = 1 << 40        # a workspace size no check refuses
NO_GPU = not torch.cuda.is_available()
OK, EINVAL, ESHAPE, EALIGN, EWS, EDEV = 0, 1, 2, 3, 4, 6
BF, F16, F32 = 0, 1, 2


def test_exports_match_header():
    text = open(HEADER).read()
    names = set(re.findall(r"MOE_API\s+[\w\s\*]+?\b(moe_\w+)\s*\(", text))
    assert names == set(_block.EXPORTS)
    for n in names:
        assert hasattr(LIB, n), n


def mm(rows=4, K=64, N=32, E=4, x_rows=4, topk=2, dtype=BF, act=0):
    return _block.MoeMMShape(rows, K, N, E, x_rows, topk, dtype, act)


BAD_SHAPES = [
    (dict(rows=-1), EINVAL), (dict(K=0), ESHAPE), (dict(K=12), ESHAPE), (dict(K=-8), ESHAPE),
    (dict(N=0), ESHAPE), (dict(N=20), ESHAPE), (dict(N=24, act=4), ESHAPE),
    (dict(dtype=2), EINVAL), (dict(dtype=-1), EINVAL), (dict(act=5), EINVAL), (dict(act=-1), EINVAL),
    (dict(K=(1 << 20) + 8), ESHAPE), (dict(N=(1 << 20) + 8), ESHAPE),
    (dict(N=1 << 16, K=1 << 15), ESHAPE),                       # N*K = 2^31
    (dict(rows=(1 << 31) - 1, N=1 << 10), ESHAPE),              # rows*N above 2^38
    (dict(rows=(1 << 31) - 1, K=8, N=16), ESHAPE), (dict(rows=(1 << 31) - 65535, K=8, N=16), ESHAPE),
]


def grouped(s, x=A, w=A, off=A, slot=None, z=None, y=A, yt=BF):
    return LIB.moe_grouped_mm(ctypes.byref(s) if s else None, *place(x, w, off, slot, z, y), yt, None)


def grouped_bwd(s, dy=A, x=A, w=A, z=None, off=A, slot=None, dx=A, dxt=BF, dw=A, dwt=BF, ws=A, n=BIG):
    dy, x, w, z, off, slot, dx, dw, ws = place(dy, x, w, z, off, slot, dx, dw, ws)
    return LIB.moe_grouped_mm_backward(ctypes.byref(s) if s else None, dy, x, w, z, off, slot, dx,
                                       dxt, dw, dwt, ws, n, None)


def lin(s, x=A, w=A, bias=None, res=None, z=None, y=A, yt=BF):
    return LIB.moe_linear(ctypes.byref(s) if s else None, *place(x, w, bias, res, z, y), yt, None)


def lin_bwd(s, dy=A, dyt=BF, x=A, w=A, z=None, dx=A, dxt=BF, dw=A, db=A, dwt=BF, ws=A, n=BIG):
    dy, x, w, z, dx, dw, db, ws = place(dy, x, w, z, dx, dw, db, ws)
    return LIB.moe_linear_backward(ctypes.byref(s) if s else None, dy, dyt, x, w, z, dx, dxt, dw,
                                   db, dwt, ws, n, None)


@pytest.mark.parametrize("change,status", BAD_SHAPES)
def test_product_shapes_refused(change, status):
    s = mm(**change)
    for f in (grouped, grouped_bwd, lin, lin_bwd):
        assert f(s) == status, f.__name__
        assert LIB.moe_last_error()
    assert LIB.moe_grouped_mm_backward_workspace(ctypes.byref(s)) == 0
    assert LIB.moe_linear_backward_workspace(ctypes.byref(s)) == 0


def test_products_refuse_null_shape():
    for f in (grouped, grouped_bwd, lin, lin_bwd):
        assert f(None) == EINVAL
    assert LIB.moe_grouped_mm_backward_workspace(None) == 0


def test_grouped_refusals():
    s = mm()
    for E in (0, 1025):
        assert grouped(mm(E=E)) == ESHAPE and grouped_bwd(mm(E=E)) == ESHAPE
    for p in ("x", "w", "off", "y"):
        assert grouped(s, **{p: None}) == EINVAL
        assert grouped(s, **{p: MIS}) == EALIGN
    assert grouped(s, z=MIS) == EALIGN
    assert grouped(s, slot=MIS) == EALIGN
    assert grouped(s, yt=F16) == EINVAL and grouped(s, yt=7) == EINVAL
    assert grouped(mm(topk=0), slot=A) == ESHAPE
    assert grouped(mm(x_rows=0), slot=A) == EINVAL
    assert grouped(mm(x_rows=1 << 25), slot=A) == ESHAPE       # x_rows*K above 2^30
    assert grouped(mm(rows=0), None, None, None, None, None, None) == OK
    if NO_GPU:
        assert grouped(s) == EDEV and grouped(s, slot=A, z=A, yt=F32) == EDEV


def test_grouped_backward_refusals():
    s, a = mm(), mm(act=2)
    for p in ("dy", "x", "w", "off"):
        assert grouped_bwd(s, **{p: None}) == EINVAL
        assert grouped_bwd(s, **{p: MIS}) == EALIGN
    assert grouped_bwd(s, dx=None, dw=None) == EINVAL
    assert grouped_bwd(s, dx=MIS) == EALIGN and grouped_bwd(s, dw=MIS) == EALIGN
    assert grouped_bwd(s, dxt=F16) == EINVAL and grouped_bwd(s, dwt=5) == EINVAL
    assert grouped_bwd(a, z=None) == EINVAL and grouped_bwd(a, z=MIS) == EALIGN
    assert grouped_bwd(mm(topk=0), slot=A) == ESHAPE
    need = LIB.moe_grouped_mm_backward_workspace(ctypes.byref(a))
    assert need >= 4 * 32 * 2
    assert grouped_bwd(a, z=A, n=need - 1) == EWS
    assert grouped_bwd(a, z=A, ws=None, n=need) == EINVAL
    assert grouped_bwd(a, z=A, ws=MIS, n=need) == EALIGN
    assert LIB.moe_grouped_mm_backward_workspace(ctypes.byref(s)) == 0
    assert grouped_bwd(mm(rows=0), dw=None) == OK              # nothing to do
    if NO_GPU:
        # what an absent output does not need may be NULL
        assert grouped_bwd(s, w=None, dx=None) == EDEV
        assert grouped_bwd(s, x=None, dw=None) == EDEV
        assert grouped_bwd(s, ws=None, n=0) == EDEV
        assert grouped_bwd(mm(rows=0), dy=None, x=None, w=None) == EDEV    # dw becomes zero


def test_linear_refusals():
    s = mm()
    for p in ("x", "w", "y"):
        assert lin(s, **{p: None}) == EINVAL
    for p in ("x", "w", "y", "bias", "res", "z"):
        assert lin(s, **{p: MIS}) == EALIGN
    assert lin(s, yt=F16) == EINVAL
    assert lin(mm(rows=0), None, None, None, None, None, None) == OK
    if NO_GPU:
        assert lin(s, bias=A, res=A, z=A, yt=F32) == EDEV


def test_linear_backward_refusals():
    s, a = mm(), mm(act=4)
    for p in ("dy", "x", "w"):
        assert lin_bwd(s, **{p: None}) == EINVAL
    for p in ("dy", "x", "w", "dx", "dw", "db"):
        assert lin_bwd(s, **{p: MIS}) == EALIGN
    assert lin_bwd(s, dx=None, dw=None, db=None) == EINVAL
    for p in ("dyt", "dxt", "dwt"):
        assert lin_bwd(s, **{p: F16}) == EINVAL
    assert lin_bwd(a) == EINVAL                                  # z
    need = LIB.moe_linear_backward_workspace(ctypes.byref(s))
    assert need >= 4 * 32 * 2
    assert lin_bwd(s, n=need - 1) == EWS and lin_bwd(s, ws=None) == EINVAL
    assert lin_bwd(mm(rows=0), dw=None, db=None) == OK
    if NO_GPU:
        assert lin_bwd(s, dyt=F32) == EDEV and lin_bwd(a, z=A) == EDEV


def norm(T=4, H=64, dtype=BF, r=BF, y=F32, gate=0, scale=1.0, eps=1e-6):
    return _block.MoeNormShape(T, H, dtype, r, y, gate, scale, eps)


def nf(s, r=A, y=A, wp=A, g=None, wn=A, ro=A, h=A):
    return LIB.moe_block_norm(ctypes.byref(s) if s else None, *place(r, y, wp, g, wn, ro, h), None)


def nb(s, r=A, dro=A, dh=A, y=A, wp=A, g=None, wn=A, dr=A, dy=A, dwp=A, dwn=A, dg=None, ws=A, n=BIG):
    return LIB.moe_block_norm_backward(ctypes.byref(s) if s else None,
                                       *place(r, dro, dh, y, wp, g, wn, dr, dy, dwp, dwn, dg, ws),
                                       n, None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), EINVAL), (dict(H=0), ESHAPE), (dict(H=60), ESHAPE), (dict(H=16392), ESHAPE),
    (dict(dtype=2), EINVAL), (dict(r=F16), EINVAL), (dict(y=F16), EINVAL), (dict(gate=4), EINVAL),
    (dict(eps=0.0), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(eps=float("inf")), EINVAL), (dict(scale=float("inf")), EINVAL),
])
def test_norm_shapes_refused(change, status):
    assert nf(norm(**change)) == status and nb(norm(**change)) == status


def test_norm_refusals():
    s, c = norm(), norm(gate=1)
    assert nf(None) == EINVAL and nb(None) == EINVAL
    assert nf(s, ro=None, h=None, wn=None) == EINVAL
    assert nf(s, wn=None) == EINVAL and nf(s, h=None) == EINVAL          # h and w_pre together
    assert nf(s, y=None) == EINVAL and nf(c, y=None, wp=None, ro=None) == EINVAL
    assert nf(c) == EINVAL                                                # gate missing
    assert nf(s, r=None) == EINVAL
    for p in ("r", "y", "wp", "wn", "ro", "h"):
        assert nf(s, **{p: MIS}) == EALIGN, p
    assert nf(c, g=MIS) == EALIGN
    assert nf(norm(T=0), None, A, None, None, A, A, A) == OK
    if NO_GPU:
        assert nf(s) == EDEV and nf(c, g=A) == EDEV and nf(s, y=None, wp=None, ro=None) == EDEV


def test_norm_backward_refusals():
    s, c, e = norm(), norm(gate=1), norm(gate=3)
    assert nb(s, dro=None, dh=None, wn=None, dwn=None) == EINVAL
    assert nb(s, wn=None) == EINVAL and nb(s, dh=None) == EINVAL
    assert nb(s, dh=None, wn=None) == EINVAL                              # dw_pre without dh
    assert nb(s, wp=None) == EINVAL                                       # dw_post without w_post
    assert nb(s, y=None, wp=None, dwp=None) == EINVAL                     # dy without y
    assert nb(s, dg=A) == EINVAL                                          # dgate without a gate
    assert nb(c) == EINVAL and nb(s, dr=None) == EINVAL and nb(s, r=None) == EINVAL
    for p in ("r", "dro", "dh", "y", "wp", "wn", "dr", "dy", "dwp", "dwn", "ws"):
        assert nb(s, **{p: MIS}) == EALIGN, p
    assert nb(c, g=A, dg=MIS) == EALIGN
    need = LIB.moe_block_norm_backward_workspace(4, 64)
    assert need >= 2 * 64 * 4
    assert nb(s, n=need - 1) == EWS and nb(s, ws=None) == EINVAL
    assert LIB.moe_block_norm_backward_workspace(4, 60) == 0
    assert LIB.moe_block_norm_backward_workspace(-1, 64) == 0
    if NO_GPU:
        # no sums over tokens asked for: no workspace
        assert nb(e, g=A, dg=A, dwp=None, dwn=None, ws=None, n=0) == EDEV
        assert nb(s, dh=None, wn=None, dwn=None, r=None) == EDEV


def cb(dout=A, y=A, pos=A, ids=A, w=A, T=4, H=64, E=8, k=2, dy=A, dyt=BF, dw=A, dl=A):
    dout, y, pos, ids, w, dy, dw, dl = place(dout, y, pos, ids, w, dy, dw, dl)
    return LIB.moe_combine_backward(dout, y, pos, ids, w, T, H, E, k, dy, dyt, dw, dl, None)


def test_combine_backward_refusals():
    assert cb(T=-1) == EINVAL and cb(E=0) == ESHAPE and cb(E=1025) == ESHAPE
    assert cb(k=0) == ESHAPE and cb(k=9) == ESHAPE and cb(E=64, k=33) == ESHAPE
    assert cb(H=0) == ESHAPE and cb(H=60) == ESHAPE
    assert cb(T=1 << 30, k=2) == ESHAPE
    assert cb(dy=None, dw=None, dl=None) == EINVAL and cb(dyt=3) == EINVAL
    for p in ("dout", "y", "pos", "ids", "w"):
        assert cb(**{p: None}) == EINVAL, p
    for p in ("dout", "y", "pos", "ids", "w", "dy", "dw", "dl"):
        assert cb(**{p: MIS}) == EALIGN, p
    assert cb(T=0, dout=None, y=None, pos=None, ids=None, w=None) == OK
    if NO_GPU:
        assert cb() == EDEV and cb(y=None, ids=None, dw=None, dl=None) == EDEV


# ------------------------------------------------------------------ binding --
def _t(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_shapes_types_and_layouts():
    import quantized_moe_expert_top_amd as moe
    off = torch.zeros(5, dtype=torch.int32)
    x, w, y = _t((6, 64)), _t((4, 32, 64)), _t((6, 32))
    bad = [
        lambda: moe.grouped_mm(_t((6, 56)), w, off, y),                       # K differs
        lambda: moe.grouped_mm(_t((5, 64)), w, off, y),                       # rows differ
        lambda: moe.grouped_mm(x, w, off[:4], y),                             # E + 1 offsets
        lambda: moe.grouped_mm(x, w, off.long(), y),
        lambda: moe.grouped_mm(x, w.half(), off, y),                          # mixed types
        lambda: moe.grouped_mm(x.float(), w.float(), off, y),
        lambda: moe.grouped_mm(x, w, off, _t((6, 32), torch.float16)),
        lambda: moe.grouped_mm(x, w, off, y, act="swiglu"),                   # y is N wide
        lambda: moe.grouped_mm(x, w, off, y, act="tanh"),
        lambda: moe.grouped_mm(x, w, off, _t((32, 6)).t()),                   # not contiguous
        lambda: moe.grouped_mm(x, w, off, y, sorted_slot=off),                # length
        lambda: moe.grouped_mm(x, w[0], off, y),
        lambda: moe.grouped_mm(_t((6, 64)), w, off, y, z=_t((6, 16))),
        lambda: moe.grouped_mm_backward(_t((6, 16)), x, w, off, dx=_t((6, 64))),
        lambda: moe.grouped_mm_backward(y, x, w, off, dw=_t((4, 64, 32))),
        lambda: moe.linear(x, w[0], _t((5, 32))),
        lambda: moe.linear(x, w[0], y, bias=_t((31,))),
        lambda: moe.linear(x, w[0], y, residual=_t((6, 32), torch.float32)),  # y's type
        lambda: moe.linear_backward(y, x, w[0], dw=_t((32, 64)), dbias=_t((32,), torch.float32)),
        lambda: moe.block_norm(_t((3, 64)), h=_t((3, 64)), w_pre=_t((63,))),
        lambda: moe.block_norm(_t((3, 64)), y=_t((3, 64)), r_out=_t((3, 64)), gate=_t((3,))),
        lambda: moe.block_norm(_t((3, 64)), h=_t((3, 64), torch.float16), w_pre=_t((64,))),
        lambda: moe.block_norm(_t((64,)), h=_t((64,)), w_pre=_t((64,))),
        lambda: moe.block_norm_backward(_t((3, 64)), _t((3, 64)), dr_out=_t((3, 64)), y=_t((3, 64)),
                                        gate=_t((64,)), dgate=_t((64,))),     # float32
        lambda: moe.combine_backward(_t((3, 64), torch.float32), _t((5, 64), torch.float32),
                                     torch.zeros(6, dtype=torch.int32), _t((3, 2), torch.float32),
                                     dtopk_w=_t((3, 2), torch.float32)),
        lambda: moe.combine_backward(_t((3, 64), torch.float32), None,
                                     torch.zeros(5, dtype=torch.int32), _t((3, 2), torch.float32),
                                     dy=_t((6, 64))),
    ]
    for i, f in enumerate(bad):
        try:
            f()
        except ValueError:
            continue
        pytest.fail(f"call {i} was not refused")


def test_binding_refuses_what_is_no_tensor():
    """Missing and foreign operands, numbers that do not fit, tensors without memory."""
    import quantized_moe_expert_top_amd as moe
    x, w, y = _t((2, 16)), _t((32, 16)), _t((2, 32))
    off, w3, slot = torch.zeros(2, dtype=torch.int32), w[None], torch.zeros(2, dtype=torch.int32)
    for bad in ([1.0], None, "x", 3):
        with pytest.raises(ValueError):
            moe.linear(bad, w, y)
        with pytest.raises(ValueError):
            moe.block_norm(bad, h=x)
    with pytest.raises(ValueError):
        moe.linear(x, w, None)
    with pytest.raises(ValueError):
        moe.linear(x.to("meta"), w.to("meta"), y.to("meta"))
    with pytest.raises(ValueError):
        moe.linear(x, w, y, residual=y.to("meta"))
    with pytest.raises(ValueError):
        moe.linear(x, w, y, act="tanh")
    with pytest.raises(ValueError):
        moe.grouped_mm(x, w3, off, y, sorted_slot=slot, topk=1 << 40)
    with pytest.raises(TypeError):
        moe.grouped_mm(x, w3, off, y, sorted_slot=slot, topk=1.5)
    with pytest.raises(TypeError):
        moe.block_norm(x, h=x, w_pre=w[0], eps="small")
    with pytest.raises(TypeError):
        moe.block_norm(x, h=x, w_pre=w[0], bias=w[0])


def test_overlaps_refused():
    """An output that overlaps an input or another output, by a byte or whole."""
    import quantized_moe_expert_top_amd as moe
    off = torch.zeros(2, dtype=torch.int32)
    buf = _t((16, 64))
    w = _t((64, 64))
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    calls = [
        lambda: moe.linear(buf[:8], w, buf[4:12]),
        lambda: moe.linear(buf[:8], w, buf[8:], residual=buf[7:15]),       # shifted by a row
        lambda: moe.linear(buf[:8], w, buf[8:], z=buf[8:]),
        lambda: moe.grouped_mm(buf[:8], w[None], off, _t((8, 64)), z=w[:8]),
        lambda: moe.block_norm(buf, y=_t((16, 64)), r_out=buf),
        lambda: moe.linear_backward(buf[:8], buf[8:], w, dx=_t((8, 64)), dw=w, ws=ws),
        lambda: moe.grouped_mm_backward(buf[:8], buf[8:], w[None], off, dx=buf[1:9], ws=ws),
        lambda: moe.linear_backward(buf[:8], buf[8:], w, dx=_t((8, 64)),
                                    ws=w.view(torch.uint8).reshape(-1)),
        lambda: moe.block_norm_backward(buf, buf, dr_out=_t((16, 64)), dh=_t((16, 64)), w_pre=w[0]),
    ]
    for i, f in enumerate(calls):
        with pytest.raises(moe.MoeError) as ei:
            f()
        assert ei.value.status == EINVAL and "overlaps" in str(ei.value), i
    if NO_GPU:
        with pytest.raises(moe.MoeError) as ei:       # the residual may be y itself
            moe.linear(buf[:8], w, buf[8:], residual=buf[8:])
        assert ei.value.status == EDEV


def test_binding_raises_library_errors():
    """What the shapes allow and the library refuses raises MoeError."""
    import quantized_moe_expert_top_amd as moe
    with pytest.raises(moe.MoeError) as ei:
        moe.linear(_t((2, 12)), _t((16, 12)), _t((2, 16)))
    assert ei.value.status == ESHAPE
    with pytest.raises(moe.MoeError) as ei:
        moe.linear_backward(_t((2, 16)), _t((2, 16)), _t((16, 16)), dx=_t((2, 16)))
    assert ei.value.status == EWS
    with pytest.raises(moe.MoeError) as ei:
        moe.block_norm(_t((2, 64)), y=_t((2, 64)))
    assert ei.value.status == EINVAL


def test_workspaces_grow_with_rows():
    """A workspace for the most rows serves any fewer."""
    import quantized_moe_expert_top_amd as moe
    g = torch.Generator().manual_seed(3)

    def rnd(lo, hi, step):
        v = lo * (hi / lo) ** torch.rand(1, generator=g).item()
        return max(step, int(v) // step * step)

    ladder = sorted({rnd(1, 40000, 1) for _ in range(150)} | set(range(0, 140)) | {4093, 8192, 8193})
    for _ in range(60):
        K, N, E = rnd(8, 9000, 8), rnd(16, 9000, 16), rnd(1, 256, 1)
        for act in ("none", "swiglu"):
            lin = [moe.linear_backward_workspace(r, K, N, act) for r in ladder]
            grp = [moe.grouped_mm_backward_workspace(r, K, N, E, act) for r in ladder]
            assert lin == sorted(lin), (K, N, act)
            assert grp == sorted(grp), (K, N, E, act)
    for H in (8, 512, 520, 2048, 16384):
        n = [moe.block_norm_backward_workspace(r, H) for r in ladder]
        assert n == sorted(n), H


def test_workspace_queries():
    import quantized_moe_expert_top_amd as moe
    assert moe.grouped_mm_backward_workspace(0, 64, 32, 4, "swiglu") == 0
    one = moe.linear_backward_workspace(100, 64, 32)
    assert one >= 100 * 32 * 2 + 32 * 4
    assert moe.linear_backward_workspace(100, 60, 32) == 0
    assert moe.block_norm_backward_workspace(10 ** 6, 2048) < 64 << 20   # bounded by the blocks
