"""The block operators (include/moe_block.h) on the GPU against plain 64-bit
forms: dense and grouped products with their epilogues and gradients, block
norms, combine gradients. Bounds are element by element, from the number of
roundings and the lengths of the float32 sums (block_ref.py)."""
import pytest

torch = pytest.importorskip("torch")

import block_ref as ref  # noqa: E402
from block_ref import close, rounded  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ("none", "relu", "silu", "gelu", "swiglu")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_moe_expert_top_amd as moe
    moe.load()


def _say(*a):
    print("[case]", *a, flush=True)


class Maker:
    """Random operands. guard=True puts each between rows of NaN, so that a read
    past its ends shows in the result."""

    def __init__(self, seed, guard=False):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.guard = guard

    def __call__(self, shape, dtype, scale=1.0):
        v = (torch.randn(shape, generator=self.g, device="cuda") * scale).to(dtype)
        if not self.guard:
            return v
        n = v.numel()
        pad = 4096
        big = torch.full((n + 2 * pad,), float("nan"), dtype=dtype, device="cuda")
        big[pad:pad + n] = v.reshape(-1)
        return big[pad:pad + n].view(shape)


def guarded(shape, dtype):
    """An output between canaries; check() verifies that they are untouched."""
    n = 1
    for s in shape:
        n *= s
    pad = 2048
    big = torch.full((n + 2 * pad,), 7.25, dtype=dtype, device="cuda")
    out = big[pad:pad + n].view(shape)
    out.fill_(float("nan"))

    def check(what):
        ends = torch.cat((big[:pad], big[pad + n:]))
        assert (ends == 7.25).all(), f"{what}: written outside its array"
    return out, check


def workspace(n):
    return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ linear --
SHAPES = [(1, 8, 16), (1, 4096, 64), (3, 72, 48), (16, 136, 528), (17, 2048, 64), (33, 64, 272),
          (64, 520, 128), (65, 200, 144), (130, 1032, 256), (257, 128, 528), (300, 264, 80),
          (515, 96, 2048), (1030, 520, 784)]


@pytest.mark.parametrize("rows,K,N", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_linear_forward(rows, K, N, act):
    import quantized_moe_expert_top_amd as moe
    i = SHAPES.index((rows, K, N)) + ACTS.index(act)
    t = (BF, HF)[i % 2]
    ty = (t, F32)[(i // 2) % 2]
    bias, res, save = i % 3 != 0, i % 3 != 1, i % 2 == 0
    _say("linear", rows, K, N, act, t, ty, bias, res, save)
    mk = Maker(i, guard=True)
    No = N // 2 if act == "swiglu" else N
    x, w = mk((rows, K), t), mk((N, K), t, K ** -0.5)
    b = mk((N,), t) if bias else None
    r = mk((rows, No), ty) if res else None
    y, ycheck = guarded((rows, No), ty)
    z, zcheck = guarded((rows, N), t) if save else (None, None)
    moe.linear(x, w, y, bias=b, residual=r, act=act, z=z)
    torch.cuda.synchronize()
    zr, ez = ref.product(x.double(), w.double(), None if b is None else b.double())
    yr, by = ref.epilogue(zr, ez, act, None if r is None else r.double(), ty)
    close(y, yr, by, "y")
    ycheck("y")
    if save:
        close(z, zr, rounded(zr, ez, t), "z")
        zcheck("z")


@pytest.mark.parametrize("rows,K,N", [(1, 8, 16), (3, 72, 48), (65, 200, 144), (130, 520, 256),
                                      (257, 128, 528), (1030, 264, 80), (2100, 136, 208)])
@pytest.mark.parametrize("act", ACTS)
def test_linear_backward(rows, K, N, act):
    import quantized_moe_expert_top_amd as moe
    i = rows + ACTS.index(act)
    t = (BF, HF)[i % 2]
    tdy = (t, F32)[(i // 2) % 2]
    tdx, tdw = (t, F32)[i % 3 == 0], (F32, t)[i % 3 == 1]
    _say("linear_backward", rows, K, N, act, t, tdy, tdx, tdw)
    mk = Maker(i, guard=True)
    No = N // 2 if act == "swiglu" else N
    x, w, dy = mk((rows, K), t), mk((N, K), t, K ** -0.5), mk((rows, No), tdy)
    z = mk((rows, N), t) if act != "none" else None
    dx, cx = guarded((rows, K), tdx)
    dw, cw = guarded((N, K), tdw)
    db, cb = guarded((N,), tdw)
    ws = workspace(moe.linear_backward_workspace(rows, K, N, act))
    moe.linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, act=act, z=z, ws=ws)
    torch.cuda.synchronize()
    zd = z.double() if z is not None else None
    dz, edz, e32 = ref.dz_pair(dy.double(), zd, act, t, from_t=tdy == t)
    xd, wd = x.double(), w.double()
    rdx, rdw, rdb = dz @ wd, dz.t() @ xd, dz.sum(0)
    close(dx, rdx, rounded(rdx, edz @ wd.abs() + (N + 2) * ref.F * ((dz.abs() + edz) @ wd.abs()), tdx), "dx")
    close(dw, rdw, rounded(rdw, edz.t() @ xd.abs() +
                           (rows + 2) * ref.F * ((dz.abs() + edz).t() @ xd.abs()), tdw), "dw")
    close(db, rdb, rounded(rdb, e32.sum(0) + (rows + 2) * ref.F * dz.abs().sum(0), tdw), "dbias")
    for c, n in ((cx, "dx"), (cw, "dw"), (cb, "dbias")):
        c(n)


@pytest.mark.parametrize("which", ["dx", "dw", "dbias"])
def test_linear_backward_single_outputs(which):
    """Each gradient alone equals what a call for all of them gives, bit for bit."""
    import quantized_moe_expert_top_amd as moe
    rows, K, N, t = 77, 136, 64, BF
    mk = Maker(5)
    x, w, dy, z = mk((rows, K), t), mk((N, K), t), mk((rows, N), F32), mk((rows, N), t)
    shapes = {"dx": (rows, K), "dw": (N, K), "dbias": (N,)}
    ws = workspace(moe.linear_backward_workspace(rows, K, N, "gelu"))
    every = {n: torch.empty(s, dtype=t, device="cuda") for n, s in shapes.items()}
    moe.linear_backward(dy, x, w, act="gelu", z=z, ws=ws, **every)
    one = torch.empty(shapes[which], dtype=t, device="cuda")
    moe.linear_backward(dy, x, w, act="gelu", z=z, ws=ws, **{which: one})
    torch.cuda.synchronize()
    assert torch.equal(one, every[which])


def test_backward_in_a_workspace_for_more_rows():
    """A workspace sized for the most rows serves fewer, cut contractions included."""
    import quantized_moe_expert_top_amd as moe
    K, N = 264, 4112
    need = moe.linear_backward_workspace(3000, K, N, "silu")
    big = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for rows in (3000, 946, 130, 3, 1):
        mk = Maker(rows)
        x, w, z, dy = mk((rows, K), BF), mk((N, K), BF), mk((rows, N), BF), mk((rows, N), BF)
        outs = []
        for ws in (big[:need], workspace(moe.linear_backward_workspace(rows, K, N, "silu"))):
            dx, dw, db = (torch.full(s, float("nan"), dtype=BF, device="cuda")
                          for s in ((rows, K), (N, K), (N,)))
            moe.linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, act="silu", z=z, ws=ws)
            outs.append((dx, dw, db))
        torch.cuda.synchronize()
        for a, b in zip(*outs):
            assert torch.isfinite(a).all() and torch.equal(a, b), rows
        assert (big[need:] == 0xA5).all()


def test_linear_adds_in_place():
    import quantized_moe_expert_top_amd as moe
    for rows, K, N in ((2, 264, 48), (140, 72, 272)):
        mk = Maker(rows)
        x, w, acc = mk((rows, K), BF), mk((N, K), BF), mk((rows, N), F32)
        want = torch.empty_like(acc)
        moe.linear(x, w, want, residual=acc.clone())
        moe.linear(x, w, acc, residual=acc)
        torch.cuda.synchronize()
        assert torch.equal(acc, want)


def test_linear_zero_rows():
    import quantized_moe_expert_top_amd as moe
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    w = torch.ones((32, 64), dtype=BF, device="cuda")
    y = torch.empty((0, 32), dtype=BF, device="cuda")
    moe.linear(x, w, y)
    dw = torch.full((32, 64), float("nan"), dtype=F32, device="cuda")
    db = torch.full((32,), float("nan"), dtype=F32, device="cuda")
    moe.linear_backward(y, x, w, dx=torch.empty_like(x), dw=dw, dbias=db,
                        ws=workspace(moe.linear_backward_workspace(0, 64, 32)))
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()


# ----------------------------------------------------------------- grouped --
def _offsets(sizes, first=0):
    o = [first]
    for s in sizes:
        o.append(o[-1] + s)
    return o


def _uneven(E, seed, most):
    g = torch.Generator().manual_seed(seed)
    n = torch.randint(0, most + 1, (E,), generator=g)
    n[torch.rand(E, generator=g) < 0.3] = 0
    return n.tolist()


# sizes of the experts, first row, rows behind the last expert
GROUPS = [([1], 0, 0), ([0, 0, 0], 0, 5), ([3, 0, 1, 0, 0, 7], 0, 0), ([0, 130, 0, 1, 64, 65], 2, 9),
          ([16] * 9, 0, 0), ([300, 5], 0, 1), (_uneven(40, 3, 33), 0, 3), (_uneven(128, 4, 70), 1, 1),
          (_uneven(1024, 5, 2), 0, 0), ([1] * 16 + [0] * 112, 0, 0), ([700, 1, 0, 257], 0, 0)]
MM = [(64, 48), (72, 128), (264, 272), (128, 64), (520, 144), (136, 528), (200, 80), (256, 144),
      (64, 32), (2048, 96), (328, 208)]


def _group_case(i, guard=True):
    sizes, first, behind = GROUPS[i]
    K, N = MM[i]
    off = _offsets(sizes, first)
    rows = off[-1] + behind
    return len(sizes), K, N, off, rows, Maker(100 + i, guard=guard)


def _sources(i, rows, gather, topk):
    """(sorted_slot or None, source row of each grouped row, rows of x)"""
    if not gather:
        return None, torch.arange(rows, device="cuda"), rows
    tokens = (rows + topk - 1) // topk + 1
    g = torch.Generator().manual_seed(i)
    slot = torch.randint(0, tokens * topk, (rows,), generator=g).to(torch.int32)
    return slot.cuda(), (slot // topk).long().cuda(), tokens


@pytest.mark.parametrize("i", range(len(GROUPS)))
@pytest.mark.parametrize("act", ("none", "swiglu", "silu"))
def test_grouped_forward(i, act):
    import quantized_moe_expert_top_amd as moe
    E, K, N, off, rows, mk = _group_case(i)
    v = i + ACTS.index(act)
    t, gather, save, topk = (BF, HF)[v % 2], (v // 2) % 2 == 0, v % 3 == 0, 1 + v % 3
    ty = (t, F32)[(v // 3) % 2]
    No = N // 2 if act == "swiglu" else N
    slot, src, tokens = _sources(i, rows, gather, topk)
    _say("grouped", i, E, K, N, rows, act, t, ty, gather, topk)
    x, w = mk((tokens, K), t), mk((E, N, K), t, K ** -0.5)
    y, ycheck = guarded((rows, No), ty)
    z, zcheck = guarded((rows, N), t)
    moe.grouped_mm(x, w, torch.tensor(off, dtype=torch.int32, device="cuda"), y, sorted_slot=slot,
                   topk=topk, act=act, z=z if save else None)
    torch.cuda.synchronize()
    xs = x.double()[src]
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        zr, ez = ref.product(xs[a:b], w[e].double())
        yr, by = ref.epilogue(zr, ez, act, None, ty)
        close(y[a:b], yr, by, f"y of expert {e}")
        if save:
            close(z[a:b], zr, rounded(zr, ez, t), f"z of expert {e}")
    for name, o in (("y", y), ("z", z)):
        assert torch.isnan(o[:off[0]]).all() and torch.isnan(o[off[-1]:]).all(), name
    if not save:
        assert torch.isnan(z).all()
    ycheck("y")
    zcheck("z")


@pytest.mark.parametrize("i", range(len(GROUPS)))
@pytest.mark.parametrize("act", ("none", "swiglu", "gelu"))
def test_grouped_backward(i, act):
    import quantized_moe_expert_top_amd as moe
    E, K, N, off, rows, mk = _group_case(i)
    v = i + ACTS.index(act)
    t, gather, topk = (BF, HF)[v % 2], (v // 2) % 2 == 0, 1 + v % 3
    tdx, tdw = (t, F32)[v % 3 == 0], (t, F32)[v % 3 == 1]
    No = N // 2 if act == "swiglu" else N
    slot, src, tokens = _sources(i, rows, gather, topk)
    _say("grouped_backward", i, E, K, N, rows, act, t, tdx, tdw, gather, topk)
    x, w, dy = mk((tokens, K), t), mk((E, N, K), t, K ** -0.5), mk((rows, No), t)
    z = mk((rows, N), t) if act != "none" else None
    # what lies outside the experts' rows must not reach any gradient
    dy[:off[0]] = float("nan")
    dy[off[-1]:] = float("inf")
    dx, cx = guarded((rows, K), tdx)
    dw, cw = guarded((E, N, K), tdw)
    ws = workspace(moe.grouped_mm_backward_workspace(rows, K, N, E, act))
    ws.view(torch.int8).fill_(-1)           # NaN patterns: nothing of it may count
    moe.grouped_mm_backward(dy, x, w, torch.tensor(off, dtype=torch.int32, device="cuda"), dx=dx,
                            dw=dw, sorted_slot=slot, topk=topk, act=act, z=z, ws=ws)
    torch.cuda.synchronize()
    xs = x.double()[src]
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            assert (dw[e] == 0).all(), f"dw of expert {e} without rows"
            continue
        dz, edz, _ = ref.dz_pair(dy[a:b].double(), z[a:b].double() if z is not None else None, act, t)
        wd, xd = w[e].double(), xs[a:b]
        rdx, rdw = dz @ wd, dz.t() @ xd
        close(dx[a:b], rdx, rounded(rdx, edz @ wd.abs() + (N + 2) * ref.F *
                                    ((dz.abs() + edz) @ wd.abs()), tdx), f"dx of expert {e}")
        close(dw[e], rdw, rounded(rdw, edz.t() @ xd.abs() + (b - a + 2) * ref.F *
                                  ((dz.abs() + edz).t() @ xd.abs()), tdw), f"dw of expert {e}")
    assert torch.isnan(dx[:off[0]]).all() and torch.isnan(dx[off[-1]:]).all()
    cx("dx")
    cw("dw")


def test_grouped_backward_long_gather():
    """More rows of one expert than the kernel holds source indices for at a time
    (1024), rows of other experts before and behind."""
    import quantized_moe_expert_top_amd as moe
    sizes, K, N, topk = [3, 4500, 0, 10, 2048], 72, 80, 3
    off = _offsets(sizes)
    rows = off[-1]
    mk = Maker(9, guard=True)
    slot, src, tokens = _sources(2, rows, True, topk)
    x, w, dy = mk((tokens, K), BF), mk((5, N, K), BF), mk((rows, N), BF)
    dw = torch.empty((5, N, K), dtype=F32, device="cuda")
    ws = workspace(moe.grouped_mm_backward_workspace(rows, K, N, 5))
    moe.grouped_mm_backward(dy, x, w, torch.tensor(off, dtype=torch.int32, device="cuda"), dw=dw,
                            sorted_slot=slot, topk=topk, ws=ws)
    torch.cuda.synchronize()
    xs, d = x.double()[src], dy.double()
    for e in range(5):
        a, b = off[e], off[e + 1]
        r = d[a:b].t() @ xs[a:b]
        close(dw[e], r, (b - a + 2) * ref.F * (d[a:b].abs().t() @ xs[a:b].abs()) + 1e-30, f"expert {e}")


def test_grouped_infinities_stay_in_their_rows():
    """An infinity or NaN in one row of x, or in one expert's weights, shows in
    that row or expert's rows only."""
    import quantized_moe_expert_top_amd as moe
    sizes = [5, 40, 3, 70]
    off = torch.tensor(_offsets(sizes), dtype=torch.int32, device="cuda")
    rows, K, N = sum(sizes), 136, 64
    mk = Maker(3)
    x, w = mk((rows, K), BF), mk((4, N, K), BF)
    clean = torch.empty((rows, N), dtype=BF, device="cuda")
    moe.grouped_mm(x, w, off, clean)
    x[7, 5] = float("inf")
    x[44, 1] = float("nan")
    w[2, 3, 9] = float("nan")
    y = torch.empty_like(clean)
    moe.grouped_mm(x, w, off, y)
    torch.cuda.synchronize()
    keep = torch.ones((rows, N), dtype=torch.bool, device="cuda")
    keep[7] = keep[44] = False
    keep[45:48, 3] = False
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[44]).all() and not torch.isfinite(y[7]).any()
    assert torch.isnan(y[45:48, 3]).all()


def test_grouped_clamps_bad_offsets_and_sources():
    """Offsets and sources outside the contract: no access out of bounds (guards
    intact); the host cannot see them."""
    import quantized_moe_expert_top_amd as moe
    rows, K, N, E = 50, 64, 48, 4
    mk = Maker(4)
    x, w = mk((10, K), BF), mk((E, N, K), BF)
    slot = torch.full((rows,), 10 ** 6, dtype=torch.int32, device="cuda")
    slot[::3] = -5
    off = torch.tensor([-7, 20, 12, 90, 200], dtype=torch.int32, device="cuda")
    y, check = guarded((rows, N), BF)
    moe.grouped_mm(x, w, off, y, sorted_slot=slot, topk=2)
    dw, cw = guarded((E, N, K), BF)
    dx, cx = guarded((rows, K), BF)
    ws = workspace(moe.grouped_mm_backward_workspace(rows, K, N, E))
    moe.grouped_mm_backward(mk((rows, N), BF), x, w, off, dx=dx, dw=dw, sorted_slot=slot, topk=2,
                            ws=ws)
    torch.cuda.synchronize()
    check("y")
    cw("dw")
    cx("dx")


# -------------------------------------------------------------------- norm --
NORM_H = [8, 64, 520, 1032, 2048, 2056, 4104, 7168, 8200, 16384]


def _gate(mk, kind, T, H, t):
    shape = {"none": None, "channel": (H,), "token": (T, 1), "element": (T, H)}[kind]
    return None if shape is None else mk(shape, t)


@pytest.mark.parametrize("H", NORM_H)
@pytest.mark.parametrize("kind", ["none", "channel", "token", "element"])
def test_block_norm_forward(H, kind):
    import quantized_moe_expert_top_amd as moe
    i = NORM_H.index(H) + len(kind)
    t = (BF, HF)[i % 2]
    tr, ty = (t, F32)[i % 3 == 0], (t, F32)[(i // 2) % 2]
    T = (1, 2, 5, 67)[i % 4]
    _say("block_norm", T, H, kind, t, tr, ty)
    mk = Maker(i, guard=True)
    r, y = mk((T, H), tr, 2.0), mk((T, H), ty)
    y[0] = 0            # a row of zeros is normalized to zeros
    wp = mk((H,), t) if i % 5 else None
    wn = mk((H,), t) if (i + 1) % 5 else None
    g = _gate(mk, kind, T, H, t)
    ro, c1 = guarded((T, H), tr)
    h, c2 = guarded((T, H), t)
    moe.block_norm(r, y=y, r_out=ro, h=h if wn is not None else None, w_post=wp, w_pre=wn, gate=g,
                   scale=-0.6, eps=1e-5)
    torch.cuda.synchronize()
    d = lambda v: None if v is None else v.double()  # noqa: E731
    scale, eps = torch.tensor(-0.6).double().item(), torch.tensor(1e-5).double().item()
    (rr, br), hh = ref.norm_forward(d(r), d(y), d(wp), d(wn), d(g), scale, eps, tr, t)
    close(ro, rr, br, "r_out")
    c1("r_out")
    c2("h")
    if wn is not None:
        close(h, hh[0], hh[1], "h")


@pytest.mark.parametrize("T,H", [(1, 8), (3, 2048), (9, 7168), (130, 264)])
def test_block_norm_only_before(T, H):
    """Without y: h = rms(r; w_pre)."""
    import quantized_moe_expert_top_amd as moe
    mk = Maker(T, guard=True)
    r, w = mk((T, H), F32), mk((H,), BF)
    h, c = guarded((T, H), BF)
    moe.block_norm(r, h=h, w_pre=w)
    torch.cuda.synchronize()
    eps = torch.tensor(1e-6).double().item()
    _, (hh, bh) = ref.norm_forward(r.double(), None, None, w.double(), None, 1.0, eps, F32, BF)
    close(h, hh, bh, "h")
    c("h")


@pytest.mark.parametrize("H", NORM_H)
@pytest.mark.parametrize("kind", ["none", "channel", "token", "element"])
def test_block_norm_backward(H, kind):
    import quantized_moe_expert_top_amd as moe
    i = NORM_H.index(H) + len(kind)
    t = (BF, HF)[i % 2]
    tr, ty = (t, F32)[i % 3 == 0], (t, F32)[(i // 2) % 2]
    T = (1, 2, 5, 67, 1100 if H <= 2056 else 530)[i % 5]
    wp_on, pre_on, dro_on = i % 4 != 0, i % 6 != 1, i % 6 != 2
    _say("block_norm_backward", T, H, kind, t, tr, ty, wp_on, pre_on, dro_on)
    mk = Maker(i, guard=True)
    r, y = mk((T, H), tr, 2.0), mk((T, H), ty)
    wp, wn = (mk((H,), t) if wp_on else None), (mk((H,), t) if pre_on else None)
    dro = mk((T, H), tr) if dro_on else None
    dh = mk((T, H), t) if pre_on else None
    g = _gate(mk, kind, T, H, t)
    names = {"dr": ((T, H), tr), "dy": ((T, H), ty)}
    if wp_on:
        names["dw_post"] = ((H,), F32)
    if pre_on:
        names["dw_pre"] = ((H,), F32)
    if kind != "none":
        names["dgate"] = (tuple(g.shape), t if kind == "element" else F32)
    outs = {n: guarded(*v) for n, v in names.items()}
    ws = workspace(moe.block_norm_backward_workspace(T, H))
    ws.view(torch.int8).fill_(-1)
    moe.block_norm_backward(r, dh=dh, dr_out=dro, y=y, w_post=wp, w_pre=wn, gate=g, scale=1.7,
                            eps=1e-6, ws=ws, **{n: o[0] for n, o in outs.items()})
    torch.cuda.synchronize()
    d = lambda v: None if v is None else v.double()  # noqa: E731
    scale, eps = torch.tensor(1.7).double().item(), torch.tensor(1e-6).double().item()
    want = ref.norm_backward(d(r), d(dro), d(dh), d(y), d(wp), d(wn), d(g), scale, eps)
    for n, (o, check) in outs.items():
        v, e = want["dgate_" + kind if n == "dgate" else n]
        close(o, v.reshape(o.shape), rounded(v, e, o.dtype).reshape(o.shape), n)
        check(n)


def test_block_norm_backward_only_before():
    import quantized_moe_expert_top_amd as moe
    T, H = 37, 520
    mk = Maker(8, guard=True)
    r, dh, w = mk((T, H), BF), mk((T, H), BF), mk((H,), BF)
    dr, c = guarded((T, H), BF)
    dw, cw = guarded((H,), F32)
    ws = workspace(moe.block_norm_backward_workspace(T, H))
    moe.block_norm_backward(r, dr, dh=dh, w_pre=w, dw_pre=dw, ws=ws)
    torch.cuda.synchronize()
    eps = torch.tensor(1e-6).double().item()
    want = ref.norm_backward(r.double(), None, dh.double(), None, None, w.double(), None, 1.0, eps)
    close(dr, want["dr"][0], rounded(*want["dr"], BF), "dr")
    close(dw, *want["dw_pre"], "dw_pre")
    c("dr")
    cw("dw_pre")


def test_block_norm_zero_tokens():
    import quantized_moe_expert_top_amd as moe
    H = 64
    e = torch.empty((0, H), dtype=BF, device="cuda")
    w = torch.ones(H, dtype=BF, device="cuda")
    moe.block_norm(e, h=e.clone(), w_pre=w)
    dw = torch.full((H,), float("nan"), device="cuda")
    moe.block_norm_backward(e, e.clone(), dh=e.clone(), w_pre=w, dw_pre=dw)
    torch.cuda.synchronize()
    assert (dw == 0).all()


# ------------------------------------------------------------------ combine --
@pytest.mark.parametrize("T,H,E,k", [(1, 8, 1, 1), (3, 520, 5, 2), (2, 7168, 256, 8), (64, 2048, 128, 8),
                                     (17, 1032, 1024, 32), (130, 264, 40, 5), (9, 16, 16, 13),
                                     (200, 120, 71, 9), (33, 256, 64, 16), (7, 248, 500, 31)])
@pytest.mark.parametrize("t", [BF, HF, F32])
def test_combine_backward(T, H, E, k, t):
    import quantized_moe_expert_top_amd as moe
    _say("combine_backward", T, H, E, k, t)
    mk = Maker(T + k, guard=True)
    g = torch.Generator().manual_seed(k)
    pos = torch.randperm(T * k, generator=g).to(torch.int32).cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    w = torch.softmax(mk((T, k), F32), -1)
    y, dout = mk((T * k, H), F32), mk((T, H), F32)
    dy, c1 = guarded((T * k, H), t)
    dw, c2 = guarded((T, k), F32)
    dl, c3 = guarded((T, E), F32)
    moe.combine_backward(dout, y, pos, w, dy=dy, dtopk_w=dw, topk_ids=ids, dlogits=dl)
    torch.cuda.synchronize()
    rows = y.double()[pos.long()].view(T, k, H)
    wd, dd = w.double(), dout.double()
    rdy = torch.empty((T * k, H), dtype=torch.float64, device="cuda")
    rdy[pos.long()] = (wd[:, :, None] * dd[:, None, :]).view(T * k, H)
    close(dy, rdy, rounded(rdy, ref.F * rdy.abs(), t), "dy")
    prod = rows * dd[:, None, :]
    rdw, edw = prod.sum(-1), (H + 2) * ref.F * prod.abs().sum(-1)
    close(dw, rdw, edw + 1e-30, "dtopk_w")
    mean = (wd * rdw).sum(1, keepdim=True)
    emean = (wd * edw).sum(1, keepdim=True) + (k + 2) * ref.F * (wd * rdw.abs()).sum(1, keepdim=True)
    rl = wd * (rdw - mean)
    el = wd * (edw + emean) + 4 * ref.F * wd * (rdw.abs() + mean.abs())
    full = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, ids.long(), rl)
    bound = torch.zeros_like(full).scatter_(1, ids.long(), el)
    close(dl, full, bound + 1e-30, "dlogits")
    for c, n in ((c1, "dy"), (c2, "dtopk_w"), (c3, "dlogits")):
        c(n)


def test_combine_backward_single_outputs():
    import quantized_moe_expert_top_amd as moe
    T, H, E, k = 21, 264, 16, 3
    mk = Maker(6)
    pos = torch.randperm(T * k).to(torch.int32).cuda()
    ids = torch.stack([torch.randperm(E)[:k] for _ in range(T)]).to(torch.int32).cuda()
    w, y, dout = torch.softmax(mk((T, k), F32), -1), mk((T * k, H), F32), mk((T, H), F32)
    full = [torch.empty((T * k, H), dtype=BF, device="cuda"), torch.empty((T, k), device="cuda"),
            torch.empty((T, E), device="cuda")]
    one = [torch.empty_like(v) for v in full]
    moe.combine_backward(dout, y, pos, w, dy=full[0], dtopk_w=full[1], topk_ids=ids, dlogits=full[2])
    moe.combine_backward(dout, None, pos, w, dy=one[0])
    moe.combine_backward(dout, y, pos, w, dtopk_w=one[1])
    moe.combine_backward(dout, y, pos, w, topk_ids=ids, dlogits=one[2])
    torch.cuda.synchronize()
    for a, b in zip(full, one):
        assert torch.equal(a, b)


# -------------------------------------------------------------- differences --
@pytest.mark.parametrize("act", ("silu", "gelu", "swiglu", "none"))
def test_gradients_against_differences(act):
    """dx, dw and dbias against central differences of the 64-bit forward."""
    import quantized_moe_expert_top_amd as moe
    rows, K, N, t = 3, 16, 32, HF
    mk = Maker(11)
    x, w, b = mk((rows, K), t), mk((N, K), t, 0.3), mk((N,), t)
    No = N // 2 if act == "swiglu" else N
    dy = mk((rows, No), t)
    z = torch.empty((rows, N), dtype=t, device="cuda")
    y = torch.empty((rows, No), dtype=F32, device="cuda")
    moe.linear(x, w, y, bias=b, act=act, z=z)
    dx, dw, db = (torch.empty(s, dtype=F32, device="cuda") for s in ((rows, K), (N, K), (N,)))
    moe.linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, act=act, z=None if act == "none" else z,
                        ws=workspace(moe.linear_backward_workspace(rows, K, N, act)))
    torch.cuda.synchronize()
    leaves = [v.double().cpu() for v in (x, w, b)]
    up = dy.double().cpu()

    def loss(ls):
        return (ref.act_fwd(ls[0] @ ls[1].t() + ls[2], act) * up).sum().item()

    h = 1e-5
    for n, (leaf, got) in enumerate(zip(leaves, (dx, dw, db))):
        flat, g = leaf.view(-1), got.double().cpu().view(-1)
        for at in range(0, flat.numel(), max(1, flat.numel() // 40)):
            keep = flat[at].item()
            flat[at] = keep + h
            hi = loss(leaves)
            flat[at] = keep - h
            lo = loss(leaves)
            flat[at] = keep
            diff = (hi - lo) / (2 * h)
            # the kernel differentiates at z rounded to fp16 and rounds dz: each
            # moves a term by at most 2^-11 relative (times |act''| |z| <= 2)
            terms = 32 * 4.0 * 3 * 2.0 ** -11 * (1 + leaf.abs().max().item())
            assert abs(diff - g[at].item()) <= terms * 0.25, (act, n, at, diff, g[at].item())


# ------------------------------------------------------ streams and graphs --
def _block_calls(seed):
    """One call of every entry point on fixed inputs: (list of calls, outputs)."""
    import quantized_moe_expert_top_amd as moe
    mk = Maker(seed)
    T, H, E, k, N = 37, 264, 6, 2, 144
    rows = T * k
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(rows)
    off = torch.tensor([0] + torch.cumsum(torch.bincount(flat, minlength=E), 0).tolist())
    i32 = lambda v: v.to(torch.int32).cuda()  # noqa: E731
    ids, slot, pos, off = i32(ids), i32(order), i32(pos), i32(off)
    new = lambda s, t=BF: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
    x, w, dy, z = mk((T, H), BF), mk((E, N, H), BF), mk((rows, N // 2), BF), mk((rows, N), BF)
    y, dx, dw = new((rows, N // 2)), new((rows, H)), new((E, N, H))
    w1, b1, ly, ldx, ldw, ldb = (mk((N, H), BF), mk((N,), BF), new((T, N)), new((T, H)),
                                 new((N, H), F32), new((N,), F32))
    ldy = mk((T, N), BF)
    r, yy, wv, gt = mk((T, H), BF), mk((T, H), F32), mk((H,), BF), mk((H,), BF)
    ro, h, dr, dyy, dwp, dwn, dg = (new((T, H)), new((T, H)), new((T, H)), new((T, H), F32),
                                    new((H,), F32), new((H,), F32), new((H,), F32))
    tw, ey, do = torch.softmax(mk((T, k), F32), -1), mk((rows, H), F32), mk((T, H), F32)
    cdy, cdw, cdl = new((rows, H)), new((T, k), F32), new((T, E), F32)
    ws = [workspace(moe.grouped_mm_backward_workspace(rows, H, N, E, "swiglu")),
          workspace(moe.linear_backward_workspace(T, H, N, "silu")),
          workspace(moe.block_norm_backward_workspace(T, H))]
    lz = mk((T, N), BF)

    def calls(stream=None):
        moe.grouped_mm(x, w, off, y, sorted_slot=slot, topk=k, act="swiglu", stream=stream)
        moe.grouped_mm_backward(dy, x, w, off, dx=dx, dw=dw, sorted_slot=slot, topk=k,
                                act="swiglu", z=z, ws=ws[0], stream=stream)
        moe.linear(x, w1, ly, bias=b1, act="gelu", stream=stream)
        moe.linear_backward(ldy, x, w1, dx=ldx, dw=ldw, dbias=ldb, act="silu", z=lz, ws=ws[1],
                            stream=stream)
        moe.block_norm(r, y=yy, r_out=ro, h=h, w_post=wv, w_pre=wv, gate=gt, stream=stream)
        moe.block_norm_backward(r, dr, dh=x, dr_out=r, y=yy, w_post=wv, w_pre=wv, gate=gt, dy=dyy,
                                dw_post=dwp, dw_pre=dwn, dgate=dg, ws=ws[2], stream=stream)
        moe.combine_backward(do, ey, pos, tw, dy=cdy, dtopk_w=cdw, topk_ids=ids, dlogits=cdl,
                             stream=stream)
    return calls, [y, dx, dw, ly, ldx, ldw, ldb, ro, h, dr, dyy, dwp, dwn, dg, cdy, cdw, cdl]


def _same(outs, want, what):
    for i, (a, b) in enumerate(zip(outs, want)):
        assert torch.equal(a, b), f"{what}: output {i}"


def test_two_runs_are_bitwise_equal():
    calls, outs = _block_calls(1)
    calls()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for o in outs:
        o.fill_(float("nan"))
    calls()
    torch.cuda.synchronize()
    _same(outs, want, "second run")


def test_two_streams_at_once():
    a, aout = _block_calls(1)
    b, bout = _block_calls(2)
    a()
    b()
    torch.cuda.synchronize()
    wa, wb = [o.clone() for o in aout], [o.clone() for o in bout]
    for o in aout + bout:
        o.fill_(float("nan"))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        a(stream=s1.cuda_stream)
        with torch.cuda.stream(s2):
            b()
    torch.cuda.synchronize()
    _same(aout, wa, "stream given")
    _same(bout, wb, "current stream")


def test_two_threads_at_once():
    import threading
    sets = [_block_calls(i) for i in (1, 2)]
    for calls, _ in sets:
        calls()
    torch.cuda.synchronize()
    wants = [[o.clone() for o in outs] for _, outs in sets]
    for _, outs in sets:
        for o in outs:
            o.fill_(float("nan"))
    torch.cuda.synchronize()
    errors = []

    def work(calls):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    calls()
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(calls,)) for calls, _ in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for (_, outs), want in zip(sets, wants):
        _same(outs, want, "two threads")


def test_host_tensors_are_refused():
    import quantized_moe_expert_top_amd as moe
    x, w = torch.zeros((2, 16), dtype=BF), torch.zeros((32, 16), dtype=BF)
    with pytest.raises(ValueError):
        moe.linear(x, w, torch.zeros((2, 32), dtype=BF))
    with pytest.raises(ValueError):
        moe.linear(x.cuda(), w, torch.zeros((2, 32), dtype=BF, device="cuda"))


def test_two_graphs_replayed_with_eager_work_between():
    a, aout = _block_calls(1)
    b, bout = _block_calls(2)
    a()
    b()
    torch.cuda.synchronize()
    wa, wb = [o.clone() for o in aout], [o.clone() for o in bout]
    graphs = []
    for calls in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()
        graphs.append(g)
    for _ in range(4):
        for o in aout + bout:
            o.fill_(float("nan"))
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        _same(aout, wa, "first graph")
        _same(bout, wb, "second graph")
        for o in aout:
            o.fill_(float("nan"))
        a()
        graphs[1].replay()
        torch.cuda.synchronize()
        _same(aout, wa, "eager between")
        _same(bout, wb, "second graph again")


def test_graph_reads_new_inputs_and_offsets():
    """A captured grouped product follows offsets that change between replays."""
    import quantized_moe_expert_top_amd as moe
    E, K, N, rows = 5, 72, 48, 200
    mk = Maker(12)
    x, w = mk((rows, K), BF), mk((E, N, K), BF)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    y = torch.empty((rows, N), dtype=F32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.grouped_mm(x, w, off, y)
    for sizes in ([40] * 5, [0, 200, 0, 0, 0], [1, 2, 3, 4, 5], [0] * 5, [100, 0, 0, 0, 100]):
        o = _offsets(sizes)
        off.copy_(torch.tensor(o, dtype=torch.int32))
        y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for e in range(E):
            if o[e] < o[e + 1]:
                zr, ez = ref.product(x[o[e]:o[e + 1]].double(), w[e].double())
                close(y[o[e]:o[e + 1]], zr, rounded(zr, ez, F32), f"{sizes} expert {e}")
        assert torch.isnan(y[o[-1]:]).all()


# ----------------------------------------------------- a whole block, trained --
def test_block_forward_and_backward_together():
    """Norm, router, routed experts, shared expert, combine, norm: forward through
    the entry points and every gradient back to the inputs and weights, against
    64-bit autograd with the same picks. Each bf16 rounding moves a value by at most
    2^-8 of itself. The longest path forward rounds h, g (twice), o: 4; back it
    rounds do, dy, dz, dx for each of two products and the norms: 10 more, and the
    rounded forward values enter each product: 2-norms are within 16 * 2^-8."""
    import quantized_moe_expert_top_amd as moe
    T, H, I, E, k, t = 96, 256, 64, 8, 2, BF
    R = T * k
    mk = Maker(21)
    r0, gain = mk((T, H), t), mk((H,), t, 0.1) + 1
    wpost, gate = mk((H,), t, 0.1) + 1, mk((H,), t)
    wr = mk((E, H), t, H ** -0.5)
    w13, w2 = mk((E, 2 * I, H), t, H ** -0.5), mk((E, H, I), t, I ** -0.5)
    s13, s2, sb = mk((2 * I, H), t, H ** -0.5), mk((H, I), t, I ** -0.5), mk((H,), t, 0.1)
    new = lambda s, d=t: torch.empty(s, dtype=d, device="cuda")  # noqa: E731
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731

    # forward
    h = new((T, H))
    moe.block_norm(r0, h=h, w_pre=gain)
    logits, ids, tw = new((T, E), F32), i32((T, k)), new((T, k), F32)
    moe.router_logits(h, wr, logits)
    moe.route_topk(logits, k, ids, tw)
    off, slot, pos, act, nact = i32(E + 1), i32(R), i32(R), i32(E), i32(4)
    moe.permute(ids, E, off, slot, pos, act, nact, workspace(moe.permute_workspace(T, E, k)))
    z, a = new((R, 2 * I)), new((R, I))
    moe.grouped_mm(h, w13, off, a, sorted_slot=slot, topk=k, act="swiglu", z=z)
    y = new((R, H), F32)
    moe.grouped_mm(a, w2, off, y)
    out = new((T, H), F32)
    moe.combine(y, pos, tw, out)
    sz, sa = new((T, 2 * I)), new((T, I))
    moe.linear(h, s13, sa, act="swiglu", z=sz)
    moe.linear(sa, s2, out, bias=sb, residual=out)
    r1, h1 = new((T, H)), new((T, H))
    moe.block_norm(r0, y=out, r_out=r1, h=h1, w_post=wpost, w_pre=gain, gate=gate, scale=0.5)

    # backward from gradients of r1 and h1
    dr1, dh1 = mk((T, H), t), mk((T, H), t)
    dr, dout = new((T, H)), new((T, H), F32)
    dwpost, dgain1, dgate = (new((H,), F32) for _ in range(3))
    ws = workspace(max(moe.block_norm_backward_workspace(T, H),
                       moe.linear_backward_workspace(T, H, 2 * I, "swiglu"),
                       moe.linear_backward_workspace(T, I, H),
                       moe.linear_backward_workspace(T, H, E),
                       moe.grouped_mm_backward_workspace(R, H, 2 * I, E, "swiglu"),
                       moe.grouped_mm_backward_workspace(R, I, H, E)))
    moe.block_norm_backward(r1, dr, dh=dh1, dr_out=dr1, y=out, w_post=wpost, w_pre=gain, gate=gate,
                            scale=0.5, dy=dout, dw_post=dwpost, dw_pre=dgain1, dgate=dgate, ws=ws)
    dsa, ds2, dsb = new((T, I)), new((H, I)), new((H,))
    moe.linear_backward(dout, sa, s2, dx=dsa, dw=ds2, dbias=dsb, ws=ws)
    dh_shared, ds13 = new((T, H), F32), new((2 * I, H))
    moe.linear_backward(dsa, h, s13, dx=dh_shared, dw=ds13, act="swiglu", z=sz, ws=ws)
    dyp, dtw, dlog = new((R, H)), new((T, k), F32), new((T, E), F32)
    moe.combine_backward(dout, y, pos, tw, dy=dyp, dtopk_w=dtw, topk_ids=ids, dlogits=dlog)
    da, dw2 = new((R, I)), new((E, H, I))
    moe.grouped_mm_backward(dyp, a, w2, off, dx=da, dw=dw2, ws=ws)
    dhp, dw13 = new((R, H), F32), new((E, 2 * I, H))
    moe.grouped_mm_backward(da, h, w13, off, dx=dhp, dw=dw13, sorted_slot=slot, topk=k,
                            act="swiglu", z=z, ws=ws)
    dh_routed = new((T, H), F32)
    moe.combine(dhp, pos, torch.ones((T, k), device="cuda"), dh_routed)
    dh_router, dwr = new((T, H), F32), new((E, H), F32)
    moe.linear_backward(dlog, h, wr, dx=dh_router, dw=dwr, ws=ws)
    dh = (dh_shared + dh_routed + dh_router).to(t)
    dr0, dgain0 = new((T, H)), new((H,), F32)
    moe.block_norm_backward(r0, dr0, dh=dh, dr_out=dr, w_pre=gain, dw_pre=dgain0, ws=ws)
    torch.cuda.synchronize()

    # 64 bits, the same picks
    P = {n: v.double().cpu().requires_grad_() for n, v in dict(
        r0=r0, gain=gain, wpost=wpost, gate=gate, wr=wr, w13=w13, w2=w2, s13=s13, s2=s2,
        sb=sb).items()}
    pick = ids.long().cpu()

    def rms(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w

    hh = rms(P["r0"], P["gain"])
    ww = torch.softmax(torch.gather(hh @ P["wr"].t(), 1, pick), -1)
    o = torch.zeros_like(hh)
    for e in range(E):
        ye = ref.act_fwd(hh @ P["w13"][e].t(), "swiglu") @ P["w2"][e].t()
        o = o + ye * (ww * (pick == e)).sum(1, keepdim=True)
    o = o + ref.act_fwd(hh @ P["s13"].t(), "swiglu") @ P["s2"].t() + P["sb"]
    rr = P["r0"] + 0.5 * P["gate"] * rms(o, P["wpost"])
    hn = rms(rr, P["gain"])
    ((rr * dr1.double().cpu()).sum() + (hn * dh1.double().cpu()).sum()).backward()

    tol = 16 * 2.0 ** -8
    for name, got, want in (
            ("r1", r1, rr), ("h1", h1, hn), ("dr0", dr0, P["r0"].grad),
            ("dgain", dgain0 + dgain1, P["gain"].grad), ("dw_post", dwpost, P["wpost"].grad),
            ("dgate", dgate, P["gate"].grad), ("dwr", dwr, P["wr"].grad),
            ("dw13", dw13, P["w13"].grad), ("dw2", dw2, P["w2"].grad),
            ("ds13", ds13, P["s13"].grad), ("ds2", ds2, P["s2"].grad), ("dsb", dsb, P["sb"].grad)):
        g, v = got.double().cpu(), want.detach()
        rel = ((g - v).norm() / v.norm()).item()
        assert rel <= tol, f"{name}: relative 2-norm {rel:.3g} > {tol:.3g}"


# ------------------------------------------------------- every tile geometry --
# Shapes that reach each geometry of the products (256x256, 128x256 and 256x128
# with 32-deep stages, 128x128, 64x128, 64x64, the split contraction and both
# gradients in one launch), with odd remainders in every direction.
GEOMETRIES = [
    # rows, K, N, experts (0: dense)
    (8200, 4104, 7184, 0), (2500, 264, 4112, 0), (4093, 2048, 1536, 0), (1100, 96, 2048, 0),
    (40000, 72, 80, 0), (700, 2056, 1040, 0), (8200, 4104, 7184, 3), (4000, 2056, 1040, 6),
    (9000, 1032, 2064, 3), (300, 64, 2064, 40), (12000, 520, 2064, 3), (16000, 1032, 2064, 60),
    (84, 3480, 288, 14), (123, 1976, 160, 66),
    # few results of long contractions: cut in parts, or over a block's waves
    (3, 464, 4704, 0), (946, 256, 5712, 0), (30, 2048, 4112, 0), (401, 5624, 128, 0),
    (70, 96, 2000, 0), (3698, 104, 1152, 0), (200, 2952, 112, 0),
    # one deep block per CU
    (1219, 2056, 1736, 0), (347, 6000, 3872, 0), (320, 1696, 8432, 0),
    # rows of dw that are no whole cache lines, more than the caches hold
    (25, 232, 3552, 53),
]


def _splits(rows, E, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(E, generator=g) ** 2 + 0.02
    n = (w / w.sum() * rows).long()
    n[E // 2] = 0
    n[0] += rows - 7 - int(n.sum())      # the last 7 rows belong to no expert
    return _offsets(n.tolist())


@pytest.mark.parametrize("rows,K,N,E", GEOMETRIES)
def test_every_geometry(rows, K, N, E):
    import quantized_moe_expert_top_amd as moe
    i = GEOMETRIES.index((rows, K, N, E))
    t = (BF, HF)[i % 2]
    act = ("swiglu", "none")[i % 2]
    _say("geometry", rows, K, N, E, t, act)
    mk = Maker(300 + i)
    No = N // 2 if act == "swiglu" else N
    off = _splits(rows, E, i) if E else [0, rows]
    oft = torch.tensor(off, dtype=torch.int32, device="cuda")
    gather, topk = E > 0 and i % 3 != 1, 4
    slot, src, tokens = _sources(i, rows, gather, topk)
    x, dy = mk((tokens, K), t), mk((rows, No), t)
    w = mk((max(E, 1), N, K), t, K ** -0.5)
    y, ycheck = guarded((rows, No), t)
    z, zcheck = guarded((rows, N), t)
    bias = mk((N,), t) if not E else None
    res = mk((rows, No), t) if not E else None
    if E:
        moe.grouped_mm(x, w, oft, y, sorted_slot=slot, topk=topk, act=act, z=z)
    else:
        moe.linear(x, w[0], y, bias=bias, residual=res, act=act, z=z)
    torch.cuda.synchronize()
    xs = x[src]
    zz = mk((rows, N), t) if act != "none" else None
    n_ws = (moe.grouped_mm_backward_workspace(rows, K, N, E, act) if E else
            moe.linear_backward_workspace(rows, K, N, act))
    ws = workspace(n_ws)

    def grads(dx, dw):
        if E:
            moe.grouped_mm_backward(dy, x, w, oft, dx=dx, dw=dw, sorted_slot=slot, topk=topk,
                                    act=act, z=zz, ws=ws)
        else:
            moe.linear_backward(dy, x, w[0], dx=dx, dw=None if dw is None else dw[0], act=act, z=zz,
                                ws=ws)
    both, apart = [], []
    for outs, calls in ((both, ((1, 1),)), (apart, ((1, 0), (0, 1)))):
        dx, cx = guarded((rows, K), t)
        dw, cw = guarded((max(E, 1), N, K), t)
        for want_dx, want_dw in calls:
            grads(dx if want_dx else None, dw if want_dw else None)
        torch.cuda.synchronize()
        cx("dx")
        cw("dw")
        outs.extend((dx, dw))
    for e in range(max(E, 1)):
        a, b = off[e], off[e + 1]
        if a == b:
            assert (both[1][e] == 0).all() and (apart[1][e] == 0).all()
            continue
        xd, wd = xs[a:b].double(), w[e].double()
        zr, ez = ref.product(xd, wd, None if bias is None else bias.double())
        yr, by = ref.epilogue(zr, ez, act, None if res is None else res.double(), t)
        close(z[a:b], zr, rounded(zr, ez, t), f"z of expert {e}")
        close(y[a:b], yr, by, f"y of expert {e}")
        del zr, ez, yr, by
        dz, edz, _ = ref.dz_pair(dy[a:b].double(), zz[a:b].double() if zz is not None else None, act, t)
        rdx, mdx = dz @ wd, (dz.abs() + edz) @ wd.abs()
        bdx = rounded(rdx, edz @ wd.abs() + (N + 2) * ref.F * mdx, t)
        rdw, mdw = dz.t() @ xd, (dz.abs() + edz).t() @ xd.abs()
        bdw = rounded(rdw, edz.t() @ xd.abs() + (b - a + 2) * ref.F * mdw, t)
        for dx, dw in (both, apart):
            close(dx[a:b], rdx, bdx, f"dx of expert {e}")
            close(dw[e], rdw, bdw, f"dw of expert {e}")
    ycheck("y")
    zcheck("z")
    for o in (y, z, both[0], apart[0]):
        assert torch.isnan(o[off[-1]:]).all()
