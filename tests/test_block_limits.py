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


@pytest.mark.skipif(not NO_GPU, reason="would run")
@pytest.mark.parametrize("rows,K,N", [(65536, 64, 262144), (65536, 8, 262144)])
def test_tiles_are_counted_as_the_offsets_cut_them(rows, K, N):
    """1024 experts share the rows: 2^20 tiles of 64x128 or less. That every expert held
    all rows would be 2^31 of them."""
    s = shape(rows, K, N, E=1024)
    assert forward(s, True) == EDEV and backward(s, True, dw=False) == EDEV


@pytest.mark.gpu
def test_many_experts_and_many_columns():
    """The same on the GPU: 65536 rows of 1024 uneven experts x 262144 columns."""
    if NO_GPU:
        pytest.skip("no GPU")
    import quantized_moe_expert_top_amd as moe
    E, rows, K, N, t = 1024, 65536, 8, 262144, torch.bfloat16
    print("[case] many experts and columns", flush=True)
    g = torch.Generator().manual_seed(2)
    n = torch.rand(E, generator=g) ** 2
    n[::7] = 0
    n = (n / n.sum() * (rows - 5)).long()              # the last rows belong to no expert
    off = [0] + torch.cumsum(n, 0).tolist()
    gd = torch.Generator(device="cuda")
    gd.manual_seed(3)
    x = torch.randn((rows, K), generator=gd, device="cuda").to(t)
    w = torch.randn((E, N, K), generator=gd, device="cuda").to(t)
    y = torch.full((rows, N), float("nan"), dtype=t, device="cuda")
    moe.grouped_mm(x, w, torch.tensor(off, dtype=torch.int32, device="cuda"), y)
    torch.cuda.synchronize()
    for a in range(0, off[-1], 4096):
        assert not torch.isnan(y[a:min(a + 4096, off[-1])]).any(), a
    assert torch.isnan(y[off[-1]:]).all()
    for e in [i for i in range(E) if n[i]][::40] + [max(i for i in range(E) if n[i])]:
        we = w[e].double()
        for p in {off[e], off[e + 1] - 1}:
            ref = we @ x[p].double()
            mag = we.abs() @ x[p].double().abs()
            # float32 sums of K products, one rounding to bf16
            tol = (K + 2) * 2.0 ** -24 * mag + 2.0 ** -8 * ref.abs() + 2.0 ** -133
            assert ((y[p].double() - ref).abs() <= tol).all(), (e, p)


@pytest.mark.skipif(not NO_GPU, reason="would run")
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("act", [0, 2, 3, 4])
@pytest.mark.parametrize("K,N", [(8, 16), (16, 16), (128, 128), (8, 128), (128, 16)])
def test_rows_up_to_the_limit_find_a_kernel_that_fits(K, N, act, grouped):
    """A row takes at least two threads (256 x 256 columns in 512), so every count of rows
    that the shape allows has a launch, whichever kernel would be fastest."""
    for rows in ((1 << 31) - (1 << 16), (1 << 30) + 77, (1 << 29) + 1, (1 << 28) + 1, 1 << 27):
        s = shape(rows, K, N, E=3, act=act)
        assert forward(s, grouped) == EDEV, (rows, LIB.moe_last_error())
        assert backward(s, grouped) == EDEV, (rows, LIB.moe_last_error())
        assert backward(s, grouped, dw=False) == EDEV, (rows, LIB.moe_last_error())


@pytest.mark.gpu
def test_more_than_a_billion_rows():
    """2^30 rows and more of 8 columns to 16: equal rows give equal results wherever they
    stand, and those of the first period are checked."""
    if NO_GPU:
        pytest.skip("no GPU")
    import quantized_moe_expert_top_amd as moe
    period, rep, K, N, t = 65537, 16384, 8, 16, torch.bfloat16
    print("[case] a billion rows", flush=True)
    gd = torch.Generator(device="cuda")
    gd.manual_seed(5)
    xp = torch.randn((period, K), generator=gd, device="cuda").to(t)
    w = torch.randn((N, K), generator=gd, device="cuda").to(t)
    x = xp.repeat(rep, 1)
    y = torch.full((period * rep, N // 2), float("nan"), dtype=t, device="cuda")
    moe.linear(x, w, y, act="swiglu")
    torch.cuda.synchronize()
    z = xp.double() @ w.double().t()
    ez = (K + 2) * 2.0 ** -24 * (xp.double().abs() @ w.double().abs().t())
    g, u = z.chunk(2, -1)
    eg, eu = ez.chunk(2, -1)
    s = g / (1 + torch.exp(-g))
    # |silu'| <= 1.1; silu with one exp2 off by |g| 2^-24 more than 10 float32 roundings
    es = 1.1 * eg + (10 + g.abs()) * 2.0 ** -24 * s.abs()
    tol = (es * (u.abs() + eu) + s.abs() * eu) * (1 + 2.0 ** -8) + 2.0 ** -8 * (s * u).abs() + 2.0 ** -133
    first = y[:period]
    assert ((first.double() - s * u).abs() <= tol).all()
    v = y.view(rep, period, N // 2)
    for a in range(0, rep, 512):
        assert (v[a:a + 512] == first).all(), a
