"""Activations of the block products and their derivatives over the whole range of
their argument, on the GPU, against 64-bit values.

Products with an exact z (few terms, each a power of two times an operand) and
float32 results leave the activation's own error; the bias gradient of a single row
is the float32 dz itself."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_moe_expert_top_amd as moe
    moe.load()


def _say(*a):
    print("[case]", *a, flush=True)


# dz by row pieces (dense, grouped), or with column sums (dense with a bias)
@pytest.mark.parametrize("grouped,dbias", [(False, False), (False, True), (True, False)])
def test_swiglu_gradient_of_large_operands(grouped, dbias):
    """dy, gate and up so large that dy * gate or dy * up leaves float32's range while
    the gradient does not: silu and silu' of a gate of -1e30 are 0, of 80 they are 80
    and 1."""
    import quantized_moe_expert_top_amd as moe
    rows, K, No = 4, 16, 16
    _say("large operands", grouped, dbias)
    dy = torch.full((rows, No), 1e30, dtype=BF, device="cuda")
    z = torch.empty((rows, 2 * No), dtype=BF, device="cuda")
    z[:, :No], z[:, No:] = -1e30, 1e30
    dy[1], z[1, :No], z[1, No:] = 1e-10, 80.0, 1e30
    x = torch.ones((rows, K), dtype=BF, device="cuda")
    w = torch.zeros((2 * No, K), dtype=BF, device="cuda")
    for n in range(2 * No):
        w[n, n % K] = 1
    dx = torch.empty((rows, K), dtype=F32, device="cuda")
    dw = torch.empty((2 * No, K), dtype=F32, device="cuda")
    db = torch.empty((2 * No,), dtype=F32, device="cuda") if dbias else None
    if grouped:
        off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        ws = torch.empty(moe.grouped_mm_backward_workspace(rows, K, 2 * No, 1, "swiglu"),
                         dtype=torch.uint8, device="cuda")
        moe.grouped_mm_backward(dy, x, w[None], off, dx=dx, dw=dw[None], act="swiglu", z=z, ws=ws)
    else:
        ws = torch.empty(moe.linear_backward_workspace(rows, K, 2 * No, "swiglu"),
                         dtype=torch.uint8, device="cuda")
        moe.linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, act="swiglu", z=z, ws=ws)
    torch.cuda.synchronize()
    d, u = dy[1, 0].double().item(), z[1, No].double().item()
    want = torch.zeros((rows, 2 * No), dtype=torch.float64, device="cuda")
    want[1, :No], want[1, No:] = d * u, d * 80.0     # silu'(80) = 1 + 80 e^-80 + ...
    # dz: at most 16 float32 roundings and one to bf16; its sums here have two terms
    tol = 2.0 ** -8 + 32 * 2.0 ** -24
    for name, got, ref in (("dx", dx, want @ w.double()), ("dw", dw, want.t() @ x.double()),
                           ("dbias", db, want.sum(0))):
        if got is None:
            continue
        assert torch.isfinite(got).all(), f"{name}: non-finite values"
        assert ((got.double() - ref).abs() <= tol * ref.abs()).all(), name


# Error bounds in units of u = 2^-24, half a step of float32; the hardware's exp2 and
# reciprocal are within one step, 2 u.
#   e^-a    exp2 2, the correction's fma 1, the argument's own rest 0.2         3.2
#   sigmoid e^-|z| 3.2, 1 + e 1, reciprocal 2, product 1                        7.2
#   silu    sigmoid 7.2, product 1                                              8.2
#   silu'   = s (1 + z c): s 7.2, fma 1, product 1 on the value; c 7.2 on s |z| c
#   cdf     fit 1.4, t (argument 1, reciprocal 2) times the 2.46 by which t P(t)
#           moves with t, Horner's fused steps 2.9, two products 2, e 3.2      16.9
#   gelu    cdf 16.9, product 1                                                17.9
#   gelu'   cdf 16.9 on cdf; e 3.2, constant 1, product 1 on |z| pdf; fma 1
U = 2.0 ** -24


def silu64(z):
    return z / (1 + torch.exp(-z))


def silu_grad64(z):
    s, c = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))
    return s * (1 + z * c), U * (9.2 * (s * (1 + z * c)).abs() + 7.2 * s * z.abs() * c)


def cdf64(z):
    return 0.5 * torch.special.erfc(-z * 0.5 ** 0.5)


def gelu_grad64(z):
    cdf, pdf = cdf64(z), torch.exp(-z * z / 2) * (2 * torch.pi) ** -0.5
    v = cdf + z * pdf
    return v, U * (16.9 * cdf + 5.2 * z.abs() * pdf + v.abs())


def arguments(lowest, highest, n):
    """Both tails, the middle, and both sides of zero down to 1e-6."""
    g = torch.Generator().manual_seed(11)
    even = lowest + (highest - lowest) * torch.rand(n // 2, generator=g, dtype=torch.float64)
    small = 10 ** (torch.rand(n - n // 2, generator=g, dtype=torch.float64) * 6.5 - 6)
    small *= torch.randint(0, 2, small.shape, generator=g) * 2 - 1
    m, e = torch.frexp(torch.cat((even, small.clamp(lowest, highest))))
    return torch.ldexp((m * 2.0 ** 16).trunc(), e - 16)     # 16 bits: the sum of two operands


RANGE = {"silu": (-87.0, 87.0), "gelu": (-13.0, 13.0), "swiglu": (-87.0, 87.0)}


@pytest.mark.parametrize("rows", [1, 300])          # weights to registers, or tiles
@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
def test_activation_error_is_relative_to_the_result(act, t, rows):
    import quantized_moe_expert_top_amd as moe
    No, K = 4096, 8
    _say("activation", act, t, rows)
    z = arguments(*RANGE[act], No).cuda()
    hi = z.to(t)
    lo = (z - hi.double()).to(t)
    N = 2 * No if act == "swiglu" else No
    w = torch.zeros((N, K), dtype=t, device="cuda")
    w[:No, 0], w[:No, 1] = hi, lo
    u = torch.ones(No, dtype=torch.float64, device="cuda")
    if act == "swiglu":
        g = torch.Generator(device="cuda")
        g.manual_seed(4)
        w[No:, 0] = torch.randn(No, generator=g, device="cuda").to(t)
        u = w[No:, 0].double()
    x = torch.zeros((rows, K), dtype=t, device="cuda")
    x[:, :2] = 1
    y = torch.empty((rows, No), dtype=F32, device="cuda")
    moe.linear(x, w, y, act=act)
    torch.cuda.synchronize()
    z = hi.double() + lo.double()
    assert torch.equal(z, z.float().double())         # exact in the product's float32
    want = (z * cdf64(z) if act == "gelu" else silu64(z) * u)
    tol = U * {"silu": 8.2, "gelu": 17.9, "swiglu": 9.2}[act] * want.abs() + 2.0 ** -149
    err = ((y.double() - want).abs() / tol).max().item()
    assert err <= 1.0, f"error {err:.3g} times its bound"


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
def test_gradient_error_is_relative_to_the_result(act, t):
    """One row: its bias gradient in float32 is dz before it is rounded."""
    import quantized_moe_expert_top_amd as moe
    No, K = 4096, 8
    N = 2 * No if act == "swiglu" else No
    _say("gradient", act, t)
    z = torch.ones((1, N), dtype=t, device="cuda")
    z[0, :No] = arguments(*RANGE[act], No).to(t).clamp(*RANGE[act])
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    if act == "swiglu":
        z[0, No:] = torch.randn(No, generator=g, device="cuda").to(t)
    dy = torch.randn((1, No), generator=g, device="cuda")
    x = torch.zeros((1, K), dtype=t, device="cuda")
    w = torch.zeros((N, K), dtype=t, device="cuda")
    db = torch.empty((N,), dtype=F32, device="cuda")
    ws = torch.empty(moe.linear_backward_workspace(1, K, N, act), dtype=torch.uint8, device="cuda")
    moe.linear_backward(dy, x, w, dbias=db, act=act, z=z, ws=ws)
    torch.cuda.synchronize()
    d, v = dy[0].double(), z[0, :No].double()
    if act == "gelu":
        a, e = gelu_grad64(v)
        want, tol = d * a, d.abs() * (e + U * a.abs())
    else:
        a, e = silu_grad64(v)
        want, tol = d * a, d.abs() * (e + U * a.abs())
        if act == "swiglu":
            u, s = z[0, No:].double(), silu64(v)
            want = torch.cat((want * u, d * s))
            tol = torch.cat(((tol + U * (d * a).abs()) * u.abs(), 9.2 * U * (d * s).abs()))
    err = ((db.double() - want).abs() / (tol + 2.0 ** -149)).max().item()
    assert err <= 1.0, f"error {err:.3g} times its bound"


@pytest.mark.parametrize("t", [BF, HF])
def test_range_of_dz(t):
    """A float32 dy enters dx and dw rounded to the operands' type, with its range (in
    fp16 under 2^-25 zero, from 65520 on infinite; both ends of the range exact), and the
    bias gradient as it is."""
    import quantized_moe_expert_top_amd as moe
    values = [2.0 ** -24, 2.0 ** -26, 65504.0, 65520.0, 2.0 ** 100, 2.0 ** -100, 0.0, 1.0]
    N = K = 16
    _say("range of dz", t)
    dy = torch.tensor(values, device="cuda").view(-1, 1).repeat(1, N)
    rows = dy.shape[0]
    w = torch.zeros((N, K), dtype=t, device="cuda")
    w[0, 0] = 1          # dx[:, 0] = dz[:, 0] + 0 dz[:, 1] + ..., NaN where dz is infinite
    x = torch.zeros((rows, K), dtype=t, device="cuda")
    dx = torch.empty((rows, K), dtype=F32, device="cuda")
    db = torch.empty((N,), dtype=F32, device="cuda")
    ws = torch.empty(moe.linear_backward_workspace(rows, K, N), dtype=torch.uint8, device="cuda")
    moe.linear_backward(dy, x, w, dx=dx, dbias=db, ws=ws)
    torch.cuda.synchronize()
    want = (dy.to(t).float() * w[:, 0].float()).sum(1)
    assert torch.equal(dx[:, 0].nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))
    if t == HF:
        assert dx[1, 0] == 0 and dx[2, 0] == 65504 and dx[0, 0] == 2.0 ** -24
        assert torch.isnan(dx[3:5, 0]).all()
    # the sum of the eight values is 2^100 to float32's half step and seven roundings
    assert abs(db.double() - sum(values)).max() <= 8 * 2.0 ** -24 * sum(values)


@pytest.mark.parametrize("rows", [1, 300])
@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
def test_half_results_are_one_rounding_off(act, t, rows):
    """16-bit results: one rounding to them, and an exponential whose argument a is
    rounded (|a| U of the result: |z| for silu, twice z^2 / 2 for gelu)."""
    import quantized_moe_expert_top_amd as moe
    No, K = 4096, 8
    _say("half activation", act, t, rows)
    z = arguments(*RANGE[act], No).to(t).double().clamp(*RANGE[act]).cuda()
    N = 2 * No if act == "swiglu" else No
    w = torch.zeros((N, K), dtype=t, device="cuda")
    w[:No, 0] = z.to(t)
    w[No:, 0] = 1
    x = torch.zeros((rows, K), dtype=t, device="cuda")
    x[:, 0] = 1
    y = torch.empty((rows, No), dtype=t, device="cuda")
    moe.linear(x, w, y, act=act)
    torch.cuda.synchronize()
    z = w[:No, 0].double()
    want = z * cdf64(z) if act == "gelu" else silu64(z)
    a = z * z if act == "gelu" else z.abs()
    tiny = 2.0 ** -25 if t == HF else 2.0 ** -134
    tol = (torch.finfo(t).eps / 2 + (18 + a) * U * (1 + 2.0 ** -8)) * want.abs() + tiny
    err = ((y.double() - want).abs() / tol).max().item()
    assert err <= 1.0, f"error {err:.3g} times its bound"


@pytest.mark.parametrize("ty", [BF, F32])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "swiglu"])
def test_activations_of_infinities_and_nan(act, ty):
    """What the formulas give in IEEE arithmetic: +infinity stays, silu and gelu of
    -infinity and their derivatives at both infinities are 0 times infinity; a NaN stays,
    and the neighbours of all of them are what they are without."""
    import quantized_moe_expert_top_amd as moe
    inf, nan = float("inf"), float("nan")
    zs = [1.5, inf, -inf, nan, -2.0, 0.0, -0.0, 3e38]
    K, No = 8, 8
    _say("infinities", act, ty)
    N = 16 if act == "swiglu" else 8
    w = torch.zeros((N, K), dtype=BF, device="cuda")
    w[:, 0] = 1
    w[:8, 0] = torch.tensor(zs)
    x = torch.zeros((3, K), dtype=BF, device="cuda")
    x[:, 0] = 1
    y = torch.empty((3, No), dtype=ty, device="cuda")
    moe.linear(x, w, y, act=act)
    zt = torch.tensor(zs, dtype=torch.float64)
    zt = zt.to(BF).double()
    want = {"relu": zt.clamp(min=0), "gelu": zt * cdf64(zt)}.get(act, silu64(zt))
    got = y.double().cpu()
    tol = (2.0 ** -8 if ty == BF else 40 * U)
    for row in got:
        for g, v, z in zip(row.tolist(), want.tolist(), zs):
            if act != "relu" and z == -inf:
                assert g != g, (z, g)
            elif v != v or abs(v) == inf:
                assert str(g) == str(v), (z, g, v)
            else:
                assert abs(g - v) <= tol * abs(v), (z, g, v)
    # derivatives, by the bias gradient of one row
    zz = torch.ones((1, N), dtype=BF, device="cuda")
    zz[0, :8] = torch.tensor(zs)
    db = torch.empty((N,), dtype=ty, device="cuda")
    ws = torch.empty(moe.linear_backward_workspace(1, K, N, act), dtype=torch.uint8, device="cuda")
    moe.linear_backward(torch.ones((1, No), dtype=BF, device="cuda"), x[:1], w, dbias=db, act=act,
                        z=zz, ws=ws)
    torch.cuda.synchronize()
    s = 1 / (1 + torch.exp(-zt))
    want = {"relu": torch.where(zt > 0, 1.0, torch.where(zt.isnan(), zt, 0.0)),
            "gelu": gelu_grad64(zt)[0]}.get(act, s * (1 + zt / (1 + torch.exp(zt))))
    for g, v, z in zip(db[:8].double().tolist(), want.tolist(), zs):
        if z != z or (act != "relu" and abs(z) == inf):
            assert g != g, (z, g)
        else:
            assert abs(g - v) <= tol * max(abs(v), 1.0), (z, g, v)


@pytest.mark.parametrize("tb", [BF, F32])
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
def test_a_bias_gradient_leaves_the_other_gradients_bits(act, tb):
    """dx and dw are the same bits with a bias gradient of either type and without."""
    import quantized_moe_expert_top_amd as moe
    rows, K, N, t = 2051, 72, 1040, BF
    _say("bits beside a bias gradient", act, tb)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(t)

    No = N // 2 if act == "swiglu" else N
    x, w, dy, z = rand(rows, K), rand(N, K), rand(rows, No), 3 * rand(rows, N)
    ws = torch.empty(moe.linear_backward_workspace(rows, K, N, act), dtype=torch.uint8, device="cuda")
    db = torch.empty((N,), dtype=tb, device="cuda")
    got = []
    for with_db in (False, True):
        dx = torch.empty((rows, K), dtype=F32, device="cuda")
        dw = torch.empty((N, K), dtype=tb, device="cuda")
        moe.linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db if with_db else None, act=act, z=z, ws=ws)
        torch.cuda.synchronize()
        got.append((dx, dw))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
