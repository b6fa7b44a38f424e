"""The block operators on arrays past 2^31 values and 2^32 bytes, and on more rows
than one launch holds. Operands repeat with a short period, so that every row's
result equals the one a period before it, bit for bit, and the first period is
checked against the plain form in 64 bits (or a short call, which other tests
check)."""
import pytest

torch = pytest.importorskip("torch")

import block_ref as ref  # noqa: E402
from block_ref import close, rounded  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_moe_expert_top_amd as moe
    moe.load()
    yield
    torch.cuda.empty_cache()


def rand(seed, shape, dtype, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def nan(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def periodic(v, period, what):
    """Every period of v's rows equals the first; returns the first."""
    v = v.view(-1, period, v.shape[-1])
    for i in range(0, v.shape[0], 64):
        assert torch.equal(v[i:i + 64], v[:1].expand(min(64, v.shape[0] - i), -1, -1)), (what, i)
    return v[0]


P, REP, WIDE = 1031, 255, 8192        # 262905 rows x 8192: 2.15e9 values, 4.3e9 bytes


def test_linear_long_inputs_and_outputs():
    import quantized_moe_expert_top_amd as moe
    narrow = 64
    x, w = rand(1, (P, WIDE), BF), rand(2, (narrow, WIDE), BF)
    y = nan((P * REP, narrow), BF)
    moe.linear(x.repeat(REP, 1), w, y)
    z, ez = ref.product(x.double(), w.double())
    close(periodic(y, P, "long x"), z, rounded(z, ez, BF), "long x")
    del y
    x, w = rand(3, (P, narrow), BF), rand(4, (WIDE, narrow), BF)
    y, zz = nan((P * REP, WIDE), BF), nan((P * REP, WIDE), BF)
    res = rand(5, (P, WIDE), BF)
    moe.linear(x.repeat(REP, 1), w, y, residual=res.repeat(REP, 1), act="relu", z=zz)
    z, ez = ref.product(x.double(), w.double())
    close(periodic(zz, P, "long z"), z, rounded(z, ez, BF), "long z")
    v, bound = ref.epilogue(z, ez, "relu", res.double(), BF)
    close(periodic(y, P, "long y"), v, bound, "long y")


def test_linear_backward_long():
    import quantized_moe_expert_top_amd as moe
    K, rows = 64, P * REP
    x, w, dy = rand(6, (P, K), BF), rand(7, (WIDE, K), BF), rand(8, (P, WIDE), BF)
    zf = rand(9, (P, WIDE), BF)
    dx, dw, db = nan((rows, K), F32), nan((WIDE, K), F32), nan((WIDE,), F32)
    ws = torch.empty(moe.linear_backward_workspace(rows, K, WIDE, "relu"), dtype=torch.uint8,
                     device="cuda")
    moe.linear_backward(dy.repeat(REP, 1), x.repeat(REP, 1), w, dx=dx, dw=dw, dbias=db, act="relu",
                        z=zf.repeat(REP, 1), ws=ws)
    dz = torch.where(zf > 0, dy, torch.zeros_like(dy)).double()
    v, e = ref.product(dz, w.double().t())
    close(periodic(dx, P, "dx"), v, rounded(v, e, F32), "dx")
    v = dz.t() @ x.double() * REP
    close(dw, v, (rows + 3) * ref.F * REP * (dz.abs().t() @ x.double().abs()), "dw")
    close(db, dz.sum(0) * REP, (rows + 3) * ref.F * REP * dz.abs().sum(0), "dbias")
    del ws, dx
    x, w, dy = rand(10, (P, WIDE), BF), rand(11, (K, WIDE), BF), rand(12, (P, K), BF)
    dx, dw = nan((rows, WIDE), BF), nan((K, WIDE), F32)
    ws = torch.empty(moe.linear_backward_workspace(rows, WIDE, K), dtype=torch.uint8, device="cuda")
    moe.linear_backward(dy.repeat(REP, 1), x.repeat(REP, 1), w, dx=dx, dw=dw, ws=ws)
    v, e = ref.product(dy.double(), w.double().t())
    close(periodic(dx, P, "wide dx"), v, rounded(v, e, BF), "wide dx")
    v = dy.double().t() @ x.double() * REP
    close(dw, v, (rows + 3) * ref.F * REP * (dy.double().abs().t() @ x.double().abs()), "wide dw")


@pytest.mark.parametrize("tokens", [3, 700])   # few rows and whole tiles per expert
def test_grouped_many_weights(tokens):
    """36 experts x 8192 x 8192: 2.4e9 weights; the experts at the far end."""
    import quantized_moe_expert_top_amd as moe
    E, n = 36, 8192
    base = rand(13, (n, n), BF)
    w = base[None].repeat(E, 1, 1)
    for e in range(E):
        w[e] *= 2.0 ** (e % 3)
    sizes = [0] * E
    for e in (0, 17, E - 2, E - 1):
        sizes[e] = tokens + e % 2
    off = torch.tensor([sum(sizes[:e]) for e in range(E + 1)], dtype=torch.int32, device="cuda")
    rows = sum(sizes)
    x, dy = rand(14, (rows, n), BF), rand(15, (rows, n), BF)
    y, dx, dw = nan((rows, n), F32), nan((rows, n), F32), nan((E, n, n), BF)
    moe.grouped_mm(x, w, off, y)
    ws = torch.empty(max(16, moe.grouped_mm_backward_workspace(rows, n, n, E)), dtype=torch.uint8,
                     device="cuda")
    moe.grouped_mm_backward(dy, x, w, off, dx=dx, dw=dw, ws=ws)
    torch.cuda.synchronize()
    at = 0
    for e in range(E):
        if not sizes[e]:
            assert not dw[e].any(), e
            continue
        r = slice(at, at + sizes[e])
        at += sizes[e]
        wd = w[e].double()
        v, b = ref.product(x[r].double(), wd)
        close(y[r], v, rounded(v, b, F32), f"y of expert {e}")
        v, b = ref.product(dy[r].double(), wd.t())
        close(dx[r], v, rounded(v, b, F32), f"dx of expert {e}")
        v, b = ref.product(dy[r].double().t(), x[r].double().t())
        close(dw[e], v, rounded(v, b, BF), f"dw of expert {e}")


@pytest.mark.parametrize("H,period,rep", [(7168, 1031, 291), (8, 1031, 2100)])
def test_block_norm_long(H, period, rep):
    """300021 rows x 7168: 2.15e9 values; 2165100 rows x 8: more than 2^21 rows."""
    import quantized_moe_expert_top_amd as moe
    T = period * rep
    r, y, wp, wn = rand(16, (period, H), BF), rand(17, (period, H), BF), rand(18, (H,), BF), rand(19, (H,), BF)
    for gate in (rand(20, (period, 1), BF), rand(21, (period, H), BF)):
        outs = {}
        for k in (1, rep):
            n = period * k
            o = {"r_out": nan((n, H), BF), "h": nan((n, H), BF), "dr": nan((n, H), BF),
                 "dy": nan((n, H), BF), "dw_pre": nan((H,), F32)}
            rr, yy, gg = r.repeat(k, 1), y.repeat(k, 1), gate.repeat(k, 1)
            moe.block_norm(rr, y=yy, r_out=o["r_out"], h=o["h"], w_post=wp, w_pre=wn, gate=gg)
            ws = torch.empty(moe.block_norm_backward_workspace(n, H), dtype=torch.uint8, device="cuda")
            moe.block_norm_backward(o["r_out"], o["dr"], dh=yy, dr_out=rr, y=yy, w_post=wp, w_pre=wn,
                                    gate=gg, dy=o["dy"], dw_pre=o["dw_pre"], ws=ws)
            outs[k] = o
        for name in ("r_out", "h", "dr", "dy"):
            assert torch.equal(periodic(outs[rep][name], period, name), outs[1][name]), name
        ro = outs[1]["r_out"].double()
        q = (ro.square().mean(1, keepdim=True) + 1e-6).rsqrt()
        terms = y.double() * ro * q
        # q: the mean's sum over H, and a dozen single roundings
        close(outs[rep]["dw_pre"], terms.sum(0) * rep,
              (T + H + 16) * ref.F * rep * terms.abs().sum(0), "dw_pre")


@pytest.mark.parametrize("T,H,k,period", [(33033, 8192, 8, 33), ((1 << 22) + 21, 8, 1, 25)])
def test_combine_backward_long(T, H, k, period):
    """33033 tokens x 8 x 8192: 2.16e9 values; and more than 2^22 tokens."""
    import quantized_moe_expert_top_amd as moe
    rep = T // period
    assert rep * period == T
    y, dout, w = rand(22, (period * k, H), F32), rand(23, (period, H), F32), rand(24, (period, k), F32).abs()
    ids = torch.stack([torch.randperm(16)[:k] for _ in range(period)]).to(torch.int32).cuda()
    outs = {}
    for n in (1, rep):
        R = period * k * n
        o = [nan((R, H), BF), nan((period * n, k), F32), nan((period * n, 16), F32)]
        pos = torch.arange(R - 1, -1, -1, dtype=torch.int32, device="cuda")
        moe.combine_backward(dout.repeat(n, 1), y.repeat(n, 1), pos, w.repeat(n, 1), dy=o[0],
                             dtopk_w=o[1], topk_ids=ids.repeat(n, 1), dlogits=o[2])
        outs[n] = o
    for i, p in enumerate((period * k, period, period)):
        assert torch.equal(periodic(outs[rep][i], p, i), outs[1][i]), i


def test_norm_of_zero_rows_at_the_smallest_eps():
    """A row of zeros has the finite gradient e / sqrt(eps)."""
    import quantized_moe_expert_top_amd as moe
    for H in (64, 2048, 8200):
        eps, n = 1e-30, 5
        z, w, e = torch.zeros((n, H), dtype=BF, device="cuda"), rand(25, (H,), BF), rand(26, (n, H), BF)
        dr, dy = nan((n, H), F32), nan((n, H), F32)
        moe.block_norm_backward(z.float(), dr, dh=e, dr_out=e.float(), y=z.float(), w_post=w, w_pre=w,
                                eps=eps, dy=dy)
        s = torch.tensor(eps).double().item() ** -0.5
        want = e.double() + s * e.double() * w.double()
        close(dr, want, 8 * ref.F * (e.double().abs() + s * (e.double() * w.double()).abs()), "dr")
        assert torch.isfinite(dr).all()
        v = want * s * w.double()
        close(dy, v, 16 * ref.F * s * (e.double().abs() + s * (e.double() * w.double()).abs()) * w.double().abs(), "dy")
