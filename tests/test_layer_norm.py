"""GPU tests of the layer norms (moe_block.h) and their gradients against plain 64-bit
forms with derived bounds, and of the gradients against differences."""
import pytest

torch = pytest.importorskip("torch")

import quantized_moe_expert_top_amd as moe  # noqa: E402
from block_ref import close, rounded  # noqa: E402
import int8_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, shape, t=F32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(t)


def operands(T, H, t, tr, ty, seed, mean=1.0):
    g = gen(seed)
    return dict(r=(randn(g, (T, H), F32, 2.0) + mean * randn(g, (T, 1))).to(tr), y=randn(g, (T, H), ty),
                w=(1 + randn(g, (H,), F32, 0.2)).to(t), b=randn(g, (H,), t, 0.3),
                dh=randn(g, (T, H), t), dr_out=randn(g, (T, H), tr))


def d(v):
    return None if v is None else v.double()


def check_forward(p, add, bias, eps=1e-5):
    T, H = p["r"].shape
    t, tr = p["w"].dtype, p["r"].dtype
    h = torch.full((T + 1, H), 9.0, dtype=t, device=DEV)
    ro = torch.full((T + 1, H), 9.0, dtype=tr, device=DEV) if add else None
    y, b = p["y"] if add else None, p["b"] if bias else None
    moe.layer_norm(p["r"], p["w"], h[:T], b=b, y=y, r_out=ro[:T] if add else None, eps=eps)
    out, (v, e) = ref.layer_norm(d(p["r"]), d(y), d(p["w"]), d(b), eps, tr, t)
    close(h[:T], v, e, ("h", T, H))
    assert (h[T] == 9).all()
    if add:
        close(ro[:T], *out, ("r_out", T, H))
        assert (ro[T] == 9).all()


def check_backward(p, add, bias, eps=1e-5, sums=True):
    T, H = p["r"].shape
    tr = p["r"].dtype
    dr = torch.full((T + 1, H), 9.0, dtype=tr, device=DEV)
    dw = torch.full((H + 8,), 9.0, device=DEV) if sums else None
    db = torch.full((H + 8,), 9.0, device=DEV) if sums and bias else None
    n = moe.layer_norm_backward_workspace(T, H)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) if sums else None
    moe.layer_norm_backward(p["r"], p["w"], p["dh"], dr[:T], dr_out=p["dr_out"] if add else None,
                            dw=dw[:H] if sums else None, db=db[:H] if db is not None else None, eps=eps,
                            ws=ws)
    want = ref.layer_norm_backward(d(p["r"]), d(p["dr_out"]) if add else None, d(p["dh"]), d(p["w"]), eps)
    v, e = want["dr"]
    close(dr[:T], v, rounded(v, e, tr), ("dr", T, H))
    assert (dr[T] == 9).all()
    if sums:
        close(dw[:H], *want["dw"], ("dw", T, H))
        assert (dw[H:] == 9).all()
    if db is not None:
        close(db[:H], *want["db"], ("db", T, H))
        assert (db[H:] == 9).all()


SIZES = [(1, 8), (3, 64), (2, 504), (9, 512), (5, 520), (3, 1024), (4, 1032), (2, 2048), (7, 2056),
         (3, 4096), (2, 4104), (2, 7168), (3, 8192), (2, 8200), (3, 16384), (4099, 64), (1537, 768),
         (900, 2048), (600, 4096), (300, 8192), (260, 16376)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("t", [BF, HF])
def test_forward(T, H, t):
    n = T + H // 8
    p = operands(T, H, t, (t, F32)[n % 2], (F32, t)[n % 3 == 0], n)
    check_forward(p, True, n % 5 != 0)
    check_forward(p, False, n % 5 == 0)


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("t", [BF, HF])
def test_backward(T, H, t):
    n = T + H // 8
    p = operands(T, H, t, (F32, t)[n % 2], t, n + 1)
    check_backward(p, True, True)
    check_backward(p, False, n % 2 == 0)
    check_backward(p, n % 2 == 0, True, sums=False)


@pytest.mark.parametrize("tr", [BF, F32])
@pytest.mark.parametrize("ty", [BF, F32])
def test_types(tr, ty):
    for T, H in ((5, 256), (3, 1536)):
        p = operands(T, H, BF, tr, ty, H)
        check_forward(p, True, True)
        check_backward(p, True, True)


@pytest.mark.parametrize("H", [64, 2048, 8192])
def test_rows_with_a_large_mean(H):
    """What a difference of squares would lose: rows of mean 1000 and deviation 2."""
    p = operands(4, H, BF, F32, F32, H, mean=0.0)
    p["r"] += 1000.0
    check_forward(p, False, True)
    check_backward(p, False, True)


@pytest.mark.parametrize("H", [64, 1024, 9000])
def test_constant_and_bad_rows(H):
    p = operands(6, H, BF, F32, F32, H)
    p["r"][0] = 0.0
    p["r"][1] = 3.0
    h = torch.empty((6, H), dtype=BF, device=DEV)
    moe.layer_norm(p["r"], p["w"], h, b=p["b"])
    assert torch.equal(h[0], p["b"]) and torch.equal(h[1], p["b"])
    check_backward(p, True, True)
    good = h.clone()
    p["r"][2, 5], p["r"][3, H - 1] = float("inf"), float("nan")
    moe.layer_norm(p["r"], p["w"], h, b=p["b"])
    assert torch.isnan(h[2]).all() and torch.isnan(h[3]).all()
    assert torch.equal(h[[0, 1, 4, 5]], good[[0, 1, 4, 5]])


def test_empty():
    e = lambda *s, t=BF: torch.empty(s, dtype=t, device=DEV)  # noqa: E731
    moe.layer_norm(e(0, 64), e(64), e(0, 64))
    dw, db = torch.ones(64, device=DEV), torch.ones(64, device=DEV)
    moe.layer_norm_backward(e(0, 64), e(64), e(0, 64), e(0, 64), dw=dw, db=db)
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("T,H", [(3, 64), (2, 1040)])
def test_gradients_against_differences(T, H):
    """Central differences of the 64-bit forward along random directions: their own error
    is step^2 times a third derivative, which is of the gradient's size here, and the
    kernel's rounding F of a sum of T H terms."""
    p = operands(T, H, BF, F32, F32, T)
    r, w, b, dh = (d(p[n]) for n in ("r", "w", "b", "dh"))

    def loss(r, w, b):
        return (ref.layer_norm(r, None, w, b, 1e-5, F32, F32)[1][0] * dh).sum()
    dr, dw, db = torch.empty_like(p["r"]), torch.empty(H, device=DEV), torch.empty(H, device=DEV)
    ws = torch.empty(moe.layer_norm_backward_workspace(T, H), dtype=torch.uint8, device=DEV)
    moe.layer_norm_backward(p["r"], p["w"], p["dh"], dr, dw=dw, db=db, ws=ws)
    step = 1e-4
    for i, (grad, at) in enumerate(((dr, 0), (dw, 1), (db, 2))):
        v = torch.randn(grad.shape, generator=gen(i), device=DEV, dtype=torch.float64)
        plus, minus = [r, w, b], [r, w, b]
        plus[at], minus[at] = plus[at] + step * v, minus[at] - step * v
        want = (loss(*plus) - loss(*minus)) / (2 * step)
        got = (grad.double() * v).sum()
        size = (grad.double() * v).abs().sum()
        assert (got - want).abs() <= 1e-5 * size, (i, got, want)


def test_in_a_graph():
    T, H = 65, 1024
    p = operands(T, H, BF, BF, BF, 3)
    e = lambda *s, t=BF: torch.empty(s, dtype=t, device=DEV)  # noqa: E731
    o = dict(r=e(T, H), h=e(T, H), dr=e(T, H), dw=e(H, t=F32), db=e(H, t=F32))
    ws = e(moe.layer_norm_backward_workspace(T, H), t=torch.uint8)

    def call():
        moe.layer_norm(p["r"], p["w"], o["h"], b=p["b"], y=p["y"], r_out=o["r"])
        moe.layer_norm_backward(o["r"], p["w"], p["dh"], o["dr"], dr_out=p["dr_out"], dw=o["dw"],
                                db=o["db"], ws=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(3):
        p["r"].copy_(randn(gen(i + 9), (T, H), BF))
        ws.fill_(i)
        g.replay()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in o.items()}
        call()
        torch.cuda.synchronize()
        for n in o:
            assert torch.equal(got[n], o[n]), n


def test_rows_past_32_bits():
    """Offsets past 2^31 values: the last rows of a long batch."""
    T, H = (1 << 21) + 3, 1024 + 8
    r = torch.zeros((T, H), dtype=BF, device=DEV)
    p = operands(5, H, BF, BF, BF, 2)
    r[-5:] = p["r"]
    h = torch.zeros((T, H), dtype=BF, device=DEV)
    moe.layer_norm(r, p["w"], h, b=p["b"])
    v, e = ref.layer_norm(d(p["r"]), None, d(p["w"]), d(p["b"]), 1e-5, BF, BF)[1]
    close(h[-5:], v, e, "last rows")
    assert torch.equal(h[0], p["b"]) and torch.equal(h[T // 2], p["b"])
    del h
    dr, dh = torch.zeros((T, H), dtype=BF, device=DEV), torch.zeros((T, H), dtype=BF, device=DEV)
    dh[-5:] = p["dh"]
    dw, db = torch.zeros(H, device=DEV), torch.zeros(H, device=DEV)
    ws = torch.empty(moe.layer_norm_backward_workspace(T, H), dtype=torch.uint8, device=DEV)
    moe.layer_norm_backward(r, p["w"], dh, dr, dw=dw, db=db, ws=ws)
    want = ref.layer_norm_backward(d(p["r"]), None, d(p["dh"]), d(p["w"]), 1e-5)
    close(dr[-5:], want["dr"][0], rounded(*want["dr"], BF), "last rows")
    close(dw, *want["dw"], "dw")
    close(db, *want["db"], "db")
