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
