"""GPU tests of the int8 operators (moe_int8.h) against plain 64-bit forms: codes bit
for bit, products and whole layers within bounds derived from the operations' roundings."""
import pytest

torch = pytest.importorskip("torch")

import quantized_moe_expert_top_amd as moe  # noqa: E402
from block_ref import close  # noqa: E402
import int8_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, shape, t=F32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(t)


def weights(g, shape):
    return torch.randint(-128, 128, shape, generator=g, device=DEV, dtype=torch.int8)


def scales(g, shape, K):
    return (0.5 + torch.rand(shape, generator=g, device=DEV)) * (K ** -0.5 / 73)


def guarded(shape, t, fill):
    """A tensor inside a larger one: (the tensor, a check that nothing around it changed)."""
    n = 1
    for d in shape:
        n *= d
    pad = 64
    buf = torch.full((n + 2 * pad,), fill, dtype=t, device=DEV)
    before = buf.clone()

    def check():
        a, b = buf[:pad], buf[pad + n:]
        assert torch.equal(a, before[:pad]) and torch.equal(b, before[pad + n:]), "written outside"
    return buf[pad:pad + n].view(shape), check


# -------------------------------------------------------------------- codes --
def run_quant(x):
    rows, K = x.shape
    q, cq = guarded((rows, K), torch.int8, 77)
    s, cs = guarded((rows,), F32, 7.0)
    moe.quant_rows(x, q, s)
    cq()
    cs()
    return q, s


def check_codes(x):
    q, s = run_quant(x)
    rq, rs = ref.codes(x)
    assert torch.equal(torch.nan_to_num(s, nan=-1.0), torch.nan_to_num(rs, nan=-1.0))
    assert torch.equal(q.double(), rq)


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("rows,K", [(1, 8), (3, 16), (5, 504), (4, 512), (7, 520), (6, 1032), (2, 2048),
                                    (9, 2056), (3, 4104), (2, 7168), (3, 8200), (2, 65536), (1021, 64)])
def test_codes(rows, K, t):
    g = gen(rows * 131 + K)
    check_codes(randn(g, (rows, K), t, 3.0))


@pytest.mark.parametrize("t", [BF, HF, F32])
def test_codes_at_the_middle(t):
    """Quotients on and next to the middle of two whole numbers: ties to even, and the
    short form's doubtful cases."""
    s = 2.0 ** -4
    half = (torch.arange(-127, 127, device=DEV) + 0.5) * s
    x = torch.zeros((6, 512), device=DEV)
    for i, eps in enumerate((0.0, 1e-7, -1e-7, 3e-5, -3e-5, 1e-3)):
        x[i, :254] = half * (1 + eps)
        x[i, 300] = 127 * s
    check_codes(x.to(t))


def test_codes_of_extreme_rows():
    """Zeros, negative zeros, subnormal and largest values; infinities and NaN stay in
    their row."""
    x = randn(gen(5), (12, 64))
    x[0] = 0.0
    x[1] = -0.0
    x[2] = 0.0
    x[2, 5] = 1e-45                      # a scale that underflows to zero
    x[3] *= 1e-39                        # a subnormal scale
    x[4] *= 1e-37                        # its border
    x[5] = torch.linspace(-3.4e38, 3.4e38, 64, device=DEV)
    x[6, 3] = float("inf")
    x[7, 9] = float("-inf")
    x[8, 63] = float("nan")
    x[9, 0] = float("nan")
    x[9, 1] = float("inf")
    x[10] = 3e-44
    check_codes(x)
    y = x.clone()
    y[3] = y[4] = y[10] = 0
    y[5] = torch.linspace(-6.5e4, 6.5e4, 64, device=DEV)
    check_codes(y.half())
    z = x.to(BF)
    check_codes(z)


# ------------------------------------------------------------------ products --
def run_linear(M, K, N, act, x_t, out, bias, res, by_codes, seed, in_place=False):
    g = gen(seed)
    No = N // 2 if act == "swiglu" else N
    x = randn(g, (M, K), x_t)
    w, u = weights(g, (N, K)), scales(g, (N,), K)
    b = randn(g, (N,), F32, 0.3) if bias else None
    r = randn(g, (M, No), out) if res else None
    y, check = guarded((M, No), out, 3.0)
    if in_place:
        y.copy_(r)
    q, s = ref.codes(x)
    args = dict(bias=b, residual=y if in_place else r, act=act)
    if by_codes:
        moe.linear_w8a8(q.to(torch.int8), w, u, y, x_scale=s, **args)
    else:
        ws = torch.empty(moe.linear_w8a8_workspace(M, K), dtype=torch.uint8, device=DEV)
        moe.linear_w8a8(x, w, u, y, ws=ws, **args)
    check()
    v, e = ref.linear(q, s, w, u, b, r, act, out)
    close(y, v, e, (M, K, N, act, x_t, out))


ACTS = ["none", "relu", "silu", "gelu", "swiglu"]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,N", [(1, 16, 16), (1, 7168, 48), (2, 2048, 176), (5, 48, 16), (16, 528, 80),
                                   (17, 1040, 96), (31, 272, 304), (33, 4112, 32), (61, 2048, 512)])
def test_small_products(M, K, N, act):
    n = M + K + N
    run_linear(M, K, N, act, (BF, HF)[n % 2], (BF, HF, F32)[n % 3], n % 5 < 3, n % 7 < 4, n % 2 == 0, n)


@pytest.mark.parametrize("x_t", [BF, HF])
@pytest.mark.parametrize("out", [BF, HF, F32])
@pytest.mark.parametrize("bias,res", [(False, False), (True, False), (False, True), (True, True)])
def test_operand_types(x_t, out, bias, res):
    for M, K, N, act in ((3, 320, 64, "silu"), (130, 320, 96, "swiglu")):
        for by_codes in (False, True):
            run_linear(M, K, N, act, x_t, out, bias, res, by_codes, M)


# every kernel of the products, with rows, columns and contraction that its tiles do not
# divide: (rows, K, N, the plan's name)
PLANS = [(7, 4112, 56, "rows by 16"), (61, 2064, 1040, "rows by 32"), (300, 1040, 1032, "64x64"),
         (1000, 2064, 1032, "64x128"), (4097, 4112, 1544, "128x128"), (1219, 10256, 1736, "128x128 deep"),
         (9000, 1040, 1544, "128x256"), (5549, 2064, 1544, "256x256")]


@pytest.mark.parametrize("M,K,N,name", PLANS)
@pytest.mark.parametrize("act,out", [("none", F32), ("gelu", BF)])
def test_every_kernel(M, K, N, name, act, out):
    if act == "none":
        assert moe.product_plan(M, K // 2, N)["forward"] == name
    run_linear(M, K, N, act, BF, out, True, act == "none", True, M)


@pytest.mark.parametrize("M,K,N,name", PLANS)
def test_every_kernel_gated(M, K, N, name):
    run_linear(M, K, N // 16 * 16, "swiglu", HF, HF, True, True, True, M + 1)


@pytest.mark.parametrize("M,K,N,name", PLANS)
@pytest.mark.parametrize("act,out", [("relu", F32), ("swiglu", HF)])
def test_every_kernel_adds_in_place(M, K, N, name, act, out):
    run_linear(M, K, N // 16 * 16, act, HF, out, False, True, True, M + 2, in_place=True)


# sizes around those where the kernel of few rows begins and ends: codes made in the call's
# one launch up to 16384 values; 8 tiles to a block; rows in LDS; and the kernel past them
@pytest.mark.parametrize("M,K,N", [(16, 1024, 272), (16, 1040, 272), (1, 16384, 32), (1, 65536, 64), (2, 65536, 64),
                                   (16, 8192, 144), (16, 16384, 48), (3, 272, 8208), (2, 64, 32768), (2, 64, 32784),
                                   (9, 48, 32000), (17, 6160, 56), (29, 1040, 2056), (32, 2048, 2048),
                                   (32, 7168, 2064), (33, 7168, 2064)])
@pytest.mark.parametrize("act,out,by_codes", [("none", BF, False), ("swiglu", F32, True), ("silu", HF, True)])
def test_few_rows_limits(M, K, N, act, out, by_codes):
    run_linear(M, K, N // 16 * 16 if act == "swiglu" else N, act, HF, out, K < 8192, True, by_codes, M + N)


@pytest.mark.parametrize("M,K,N,act", [(40003, 65536, 16, "none"), (140003, 32, 16384, "relu"), (70003, 65536, 32, "swiglu")])
def test_arrays_past_32_bits(M, K, N, act):
    """Offsets of x, its codes and y past 2^31 and 2^32: rows at the ends and around them."""
    g = gen(M)
    w, u = weights(g, (N, K)), scales(g, (N,), K)
    q = torch.empty((M, K), dtype=torch.int8, device=DEV).random_(-127, 128, generator=g)
    sc = torch.rand((M,), generator=g, device=DEV) * 0.01
    y = torch.full((M, N // 2 if act == "swiglu" else N), 3.0, dtype=BF, device=DEV)
    moe.linear_w8a8(q, w, u, y, x_scale=sc, act=act)
    at = sorted({0, 1, M - 1, M - 2, *(min(b // n + d, M - 1) for b in (2 ** 31, 2 ** 32)
                                       for n in (K, N) for d in (0, 1))})
    v, e = ref.linear(q[at].double(), sc[at], w, u, None, None, act, BF)
    close(y[at], v, e, (M, K, N, act))


def test_codes_of_rows_past_32_bits():
    M, K = 66001, 65536
    x = torch.empty((M, K), dtype=BF, device=DEV).normal_(generator=gen(3))
    q, s = torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty((M,), device=DEV)
    moe.quant_rows(x, q, s)
    at = [0, 32767, 32768, 65535, 65536, M - 1]
    rq, rs = ref.codes(x[at])
    assert torch.equal(s[at], rs.float()) and torch.equal(q[at].double(), rq.double())


def test_largest_codes():
    """Sums at the ends of 32 bits: K 65536, every product 128 * 128 (2^30)."""
    M, K, N = 2, 65536, 16
    q = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    s, u = torch.full((M,), 2.0 ** -10, device=DEV), torch.full((N,), 2.0 ** -10, device=DEV)
    y = torch.empty((M, N), device=DEV)
    moe.linear_w8a8(q, w, u, y, x_scale=s)
    assert torch.equal(y, torch.full_like(y, 2.0 ** 10))


def test_residual_in_place_and_empty():
    run_linear(33, 64, 64, "none", BF, F32, True, True, True, 1, in_place=True)
    run_linear(3, 64, 64, "swiglu", HF, HF, False, True, False, 2, in_place=True)
    e = torch.empty
    moe.linear_w8a8(e((0, 64), dtype=BF, device=DEV), weights(gen(1), (16, 64)), scales(gen(1), (16,), 64),
                    e((0, 16), device=DEV))
    moe.quant_rows(e((0, 64), device=DEV), e((0, 64), dtype=torch.int8, device=DEV), e((0,), device=DEV))


@pytest.mark.parametrize("M", [4, 40, 300])
def test_bad_rows_stay_alone(M):
    g = gen(M)
    K, N = 512, 64
    x = randn(g, (M, K), BF)
    w, u = weights(g, (N, K)), scales(g, (N,), K)
    ws = torch.empty(moe.linear_w8a8_workspace(M, K), dtype=torch.uint8, device=DEV)
    good, y = torch.empty((M, N), device=DEV), torch.empty((M, N), device=DEV)
    moe.linear_w8a8(x, w, u, good, ws=ws)
    x[1, 3], x[3, 7], x[2] = float("inf"), float("nan"), 0.0
    moe.linear_w8a8(x, w, u, y, ws=ws)
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all() and not y[2].any()
    rest = [i for i in range(M) if i not in (1, 2, 3)]
    assert torch.equal(y[rest], good[rest])


# --------------------------------------------------------------------- layer --
def make_layer(T, H, I, E, seed, x_t=BF):
    g = gen(seed)
    return dict(logits=randn(g, (T, E)) + 0.5 * randn(g, (E,)), x=randn(g, (T, H), x_t),
                w13=weights(g, (E, 2 * I, H)), s13=scales(g, (E, 2 * I), H),
                w2=weights(g, (E, H, I)), s2=scales(g, (E, H), I))


def run_layer(p, k, out=BF, residual=None, offsets=False, ws=None, in_place=False):
    T, H = p["x"].shape
    E, I = p["w2"].shape[0], p["w2"].shape[2]
    ids, c1 = guarded((T, k), torch.int32, -5)
    w, c2 = guarded((T, k), F32, -5.0)
    o, c3 = guarded((T, H), out, -5.0)
    off, c4 = guarded((E + 1,), torch.int32, -5)
    if in_place:
        o.copy_(residual)
    if ws is None:
        n = moe.layer_w8a8_workspace(T, H, I, E, k)
        ws = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device=DEV)[:n]
    moe.layer_w8a8(p["logits"], p["x"], p["w13"], p["s13"], p["w2"], p["s2"], ids, w, o, ws,
                   residual=o if in_place else residual, expert_offsets=off if offsets else None)
    for c in (c1, c2, c3, c4):
        c()
    return ids, w, o, off


def check_layer(p, k, out=BF, residual=None, in_place=False):
    ids, w, o, off = run_layer(p, k, out, residual, True, in_place=in_place)
    rid, rw, ro, bound = ref.layer(p["logits"], p["x"], p["w13"], p["s13"], p["w2"], p["s2"], k,
                                   residual, out)
    assert torch.equal(ids.long(), rid)
    assert (w.double() - rw).abs().max() <= 1e-6
    E = p["w2"].shape[0]
    counts = torch.bincount(rid.reshape(-1), minlength=E)
    assert torch.equal(off.long(), torch.cat([counts.new_zeros(1), counts.cumsum(0)]))
    close(o, ro, bound, (p["x"].shape, E, k))


SHAPES = [(1, 16, 16, 1, 1), (1, 256, 128, 8, 2), (2, 2048, 768, 128, 8), (2, 144, 80, 5, 5),
          (3, 1040, 272, 40, 3), (4, 512, 256, 64, 8), (4, 7168, 64, 16, 4), (5, 528, 400, 130, 6),
          (8, 2064, 784, 32, 2), (13, 1024, 512, 300, 8), (16, 2048, 768, 128, 8), (17, 320, 160, 12, 4),
          (33, 256, 176, 7, 3), (64, 1024, 384, 128, 8), (100, 256, 128, 4, 1), (1, 64, 2048, 600, 32),
          (2, 48, 32, 1024, 16), (16, 16, 16, 2, 1), (300, 512, 256, 64, 8), (16, 8192, 1040, 16, 4),
          (12, 16384, 16, 3, 2), (50, 2064, 272, 64, 10), (64, 80, 48, 1000, 8), (512, 64, 32, 64, 1),
          (512, 256, 128, 4, 2), (1301, 528, 272, 8, 3)]


@pytest.mark.parametrize("T,H,I,E,k", SHAPES)
@pytest.mark.parametrize("x_t", [BF, HF])
def test_layer(T, H, I, E, k, x_t):
    p = make_layer(T, H, I, E, T * 7 + H + E, x_t)
    check_layer(p, k, x_t)
    res = randn(gen(9), (T, H), x_t)
    check_layer(p, k, x_t, residual=res, in_place=True)


@pytest.mark.parametrize("T,H,I,E,k", [(32767, 8192, 32, 8, 8), (12288, 16384, 16, 1024, 8)])
def test_layer_at_the_limit(T, H, I, E, k):
    """T k H just below 2^31, with 128-row tiles and with low ones: some of the tokens."""
    p = make_layer(T, H, I, E, 5)
    _, _, o, off = run_layer(p, k, offsets=True)
    assert int(off[E]) == T * k
    at = [0, 1, T // 2, T - 2, T - 1]
    _, _, v, bound = ref.layer(p["logits"][at], p["x"][at], p["w13"], p["s13"], p["w2"], p["s2"], k, None, BF)
    close(o[at], v, bound, (T, H, I, E, k))


@pytest.mark.parametrize("out", [BF, HF, F32])
def test_layer_out_types(out):
    for T in (2, 11, 40):
        p = make_layer(T, 256, 128, 16, T)
        check_layer(p, 4, out)
        check_layer(p, 4, out, residual=randn(gen(T), (T, 256), out))


@pytest.mark.parametrize("T", [1, 4, 9, 16, 64])
def test_layer_routing_corners(T):
    """Ties, signed zeros, every token to the same experts, every token to its own."""
    H, I, E, k = 128, 64, 96, 4
    p = make_layer(T, H, I, E, 3)
    p["logits"] = torch.zeros((T, E), device=DEV)
    p["logits"][:, ::2] = -0.0
    check_layer(p, k)
    p["logits"][:, 90:94] = 1.0
    check_layer(p, k)
    p["logits"] = torch.full((T, E), -1e30, device=DEV)
    for t in range(T):
        p["logits"][t, (torch.arange(k) + k * t) % E] = 2.0
    check_layer(p, k)


@pytest.mark.parametrize("T", [1, 3, 16, 30])
def test_layer_zero_and_bad_tokens(T):
    p = make_layer(T, 256, 128, 16, 4)
    _, _, good, _ = run_layer(p, 4, F32)
    good = good.clone()
    p["x"][0] = 0.0
    if T > 2:
        p["x"][1, 17], p["x"][2, 5] = float("inf"), float("nan")
    _, _, o, _ = run_layer(p, 4, F32)
    assert not o[0].any()
    if T > 2:
        assert torch.isnan(o[1]).all() and torch.isnan(o[2]).all()
    assert torch.equal(o[3:], good[3:])


@pytest.mark.parametrize("T,E", [(2, 16), (13, 48), (16, 600), (40, 32), (90, 16)])
def test_layer_with_bad_logits(T, E):
    """Rows of logits without an order: route_topk's picks, all of them experts; no other
    token changes by a bit."""
    p, k = make_layer(T, 256, 128, E, T), 4
    _, _, good, _ = run_layer(p, k, F32)
    good = good.clone()
    p["logits"][0] = float("nan")
    bad = [0]
    if T > 2:
        p["logits"][3] = float("-inf")
        p["logits"][5, ::2] = float("nan")
        p["logits"][7] = float("inf")
        bad += [3, 5, 7]
    ids, w, o, off = run_layer(p, k, F32, offsets=True)
    rid, rw = torch.empty_like(ids), torch.empty_like(w)
    moe.route_topk(p["logits"], k, rid, rw)
    assert torch.equal(ids, rid) and torch.equal(w.view(torch.int32), rw.view(torch.int32))
    assert int(ids.min()) >= 0 and int(ids.max()) < E
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E)
    assert torch.equal(off.long(), torch.cat([counts.new_zeros(1), counts.cumsum(0)]))
    rest = [t for t in range(T) if t not in bad]
    assert torch.equal(o[rest], good[rest])


def test_layer_is_the_separate_calls():
    """The picks and weights of route_topk, and the sums of the separate calls."""
    for T in (2, 12, 80):
        H, I, E, k = 512, 256, 32, 4
        p = make_layer(T, H, I, E, T)
        ids, w, o, off = run_layer(p, k, F32, offsets=True)
        b = moe.LayerBuffers.alloc(T, H, I, E, k, "w8a8")
        moe.moe_forward(b, p["x"], p["logits"], (p["w13"], p["s13"], p["w2"], p["s2"]))
        assert torch.equal(ids, b.ids) and torch.equal(w, b.w) and torch.equal(off, b.offsets)
        got = b.out.clone()
        moe.moe_layer(b, p["x"].view(torch.int16), p["logits"], (p["w13"], p["s13"], p["w2"], p["s2"]))
        assert torch.equal(b.out, o)
        b.out.copy_(got)
        # codes of h may differ in one step where float32 forms of h differ
        rel = (o - b.out).norm() / b.out.norm()
        assert rel < 2e-3, rel


@pytest.mark.parametrize("T", [2, 16, 24])
def test_layer_bits_repeat_and_do_not_depend_on_the_workspace(T):
    p = make_layer(T, 1024, 320, 48, 8)
    n = moe.layer_w8a8_workspace(T, 1024, 320, 48, 6)
    first = None
    for fill in (0, 255, 0x7F):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        _, _, o, _ = run_layer(p, 6, BF, ws=ws)
        first = o.clone() if first is None else first
        assert torch.equal(first.view(torch.int16), o.view(torch.int16))


# ------------------------------------------------------- streams and graphs --
@pytest.mark.parametrize("T", [1, 2, 13, 40])
def test_layer_in_a_graph(T):
    H, I, E, k = 512, 256, 32, 4
    p = make_layer(T, H, I, E, 6)
    ws = torch.empty(moe.layer_w8a8_workspace(T, H, I, E, k), dtype=torch.uint8, device=DEV)
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w, o = torch.empty((T, k), device=DEV), torch.empty((T, H), device=DEV, dtype=BF)

    def call():
        moe.layer_w8a8(p["logits"], p["x"], p["w13"], p["s13"], p["w2"], p["s2"], ids, w, o, ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(4):
        p["x"].copy_(randn(gen(50 + i), (T, H), BF))
        p["logits"].copy_(randn(gen(70 + i), (T, E)))
        ws.fill_(i)
        g.replay()
        torch.cuda.synchronize()
        got = (ids.clone(), w.clone(), o.clone())
        call()
        torch.cuda.synchronize()
        for a, b in zip(got, (ids, w, o)):
            assert torch.equal(a, b)


def test_two_graphs_on_one_workspace():
    """Nothing is kept in a workspace between calls: two graphs that share one, replayed in
    turn, give what each gives alone."""
    H, I, E, k = 512, 256, 32, 4
    rows = (3, 40, 150)   # the layer's three ways
    n = moe.layer_w8a8_workspace(max(rows), H, I, E, k)
    ws = torch.empty(max(n, moe.linear_w8a8_workspace(max(rows), H)), dtype=torch.uint8, device=DEV)
    runs = []
    for T in rows:
        p = make_layer(T, H, I, E, 40 + T)
        ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
        w, o = torch.empty((T, k), device=DEV), torch.empty((T, H), device=DEV, dtype=BF)
        y = torch.empty((T, 2 * I), device=DEV)

        def call(p=p, ids=ids, w=w, o=o, y=y):
            moe.linear_w8a8(p["x"], p["w13"][0], p["s13"][0], y, ws=ws)
            moe.layer_w8a8(p["logits"], p["x"], p["w13"], p["s13"], p["w2"], p["s2"], ids, w, o, ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((p, o, y, call, g))
    for i in range(3):
        for p, *_ in runs:
            p["x"].copy_(randn(gen(90 + i), p["x"].shape, BF))
        for *_, g in runs:
            g.replay()
        torch.cuda.synchronize()
        got = [(o.clone(), y.clone()) for _, o, y, *_ in runs]
        for (_, o, y, call, _), (go, gy) in zip(runs, got):
            call()
            torch.cuda.synchronize()
            assert torch.equal(o, go) and torch.equal(y, gy)


def test_two_streams_at_once():
    cases = []
    for i, T in enumerate((2, 16, 2, 24)):
        p = make_layer(T, 1024, 512, 64, 20 + i)
        _, _, want, _ = run_layer(p, 8)
        cases.append((p, T, want.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        for p, T, want, st in cases:
            with torch.cuda.stream(st):
                n = moe.layer_w8a8_workspace(T, 1024, 512, 64, 8)
                ws = torch.empty(n, dtype=torch.uint8, device=DEV)
                ids = torch.empty((T, 8), dtype=torch.int32, device=DEV)
                w, o = torch.empty((T, 8), device=DEV), torch.empty((T, 1024), device=DEV, dtype=BF)
                moe.layer_w8a8(p["logits"], p["x"], p["w13"], p["s13"], p["w2"], p["s2"], ids, w, o, ws)
                outs.append((o, want, ws, ids, w))
    torch.cuda.synchronize()
    for o, want, *_ in outs:
        assert torch.equal(o, want)


def block(h_in, y, W, T, H, I, E, k, buf):
    """Layer norm, router, shared expert and routed layer, each adding to the last."""
    moe.layer_norm(h_in, W["ln_w"], buf["h"], b=W["ln_b"], y=y, r_out=buf["r"])
    moe.router_logits(buf["h"], W["router"], buf["logits"])
    moe.linear_w8a8(buf["h"], W["up"], W["up_s"], buf["mid"], act="swiglu", ws=buf["ws"])
    moe.quant_rows(buf["mid"], buf["q"], buf["qs"])
    moe.linear_w8a8(buf["q"], W["down"], W["down_s"], buf["shared"], x_scale=buf["qs"])
    moe.layer_w8a8(buf["logits"], buf["h"], W["w13"], W["s13"], W["w2"], W["s2"], buf["ids"], buf["w"],
                   buf["shared"], buf["lws"], residual=buf["shared"], expert_offsets=buf["off"])


@pytest.mark.parametrize("T", [1, 2, 12, 40])
def test_block_run(T):
    """The operators together as a block uses them, eager and replayed: each against its
    64-bit form on what the one before it gave."""
    H, I, E, k, S = 512, 256, 16, 4, 384
    g = gen(T)
    W = dict(ln_w=(1 + randn(g, (H,), F32, 0.1)).to(BF), ln_b=randn(g, (H,), BF, 0.1),
             router=randn(g, (E, H), BF, H ** -0.5), up=weights(g, (2 * S, H)),
             up_s=scales(g, (2 * S,), H), down=weights(g, (H, S)), down_s=scales(g, (H,), S),
             w13=weights(g, (E, 2 * I, H)), s13=scales(g, (E, 2 * I), H), w2=weights(g, (E, H, I)),
             s2=scales(g, (E, H), I))
    e = lambda *s, t=BF: torch.empty(s, dtype=t, device=DEV)  # noqa: E731
    buf = dict(h=e(T, H), r=e(T, H), logits=e(T, E, t=F32), mid=e(T, S), q=e(T, S, t=torch.int8),
               qs=e(T, t=F32), shared=e(T, H), ids=e(T, k, t=torch.int32), w=e(T, k, t=F32),
               off=e(E + 1, t=torch.int32), ws=e(moe.linear_w8a8_workspace(T, H), t=torch.uint8),
               lws=e(moe.layer_w8a8_workspace(T, H, I, E, k), t=torch.uint8))
    r, y = randn(g, (T, H), BF, 2.0), randn(g, (T, H), BF)
    block(r, y, W, T, H, I, E, k, buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(r, y, W, T, H, I, E, k, buf)
    for i in range(3):
        r.copy_(randn(gen(i + 100), (T, H), BF, 2.0))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in buf.items()}
        block(r, y, W, T, H, I, E, k, buf)
        torch.cuda.synchronize()
        for n in ("h", "r", "logits", "mid", "q", "qs", "shared", "ids", "w", "off"):
            assert torch.equal(got[n], buf[n]), n
        (ro, rb), (h, hb) = ref.layer_norm(r.double(), y.double(), W["ln_w"].double(), W["ln_b"].double(),
                                           1e-5, BF, BF)
        close(got["r"], ro, rb, "r")
        close(got["h"], h, hb, "h")
        q, s = ref.codes(got["h"])
        v, b = ref.linear(q, s, W["up"], W["up_s"], None, None, "swiglu", BF)
        close(got["mid"], v, b, "mid")
        q, s = ref.codes(got["mid"])
        assert torch.equal(got["q"].double(), q) and torch.equal(got["qs"], s)
        shared = e(T, H)
        moe.linear_w8a8(got["q"], W["down"], W["down_s"], shared, x_scale=got["qs"])
        ids, w, o, ob = ref.layer(got["logits"], got["h"], W["w13"], W["s13"], W["w2"], W["s2"], k,
                                  shared, BF)
        assert torch.equal(got["ids"].long(), ids)
        close(got["shared"], o, ob, "out")
