"""The int8 operators and layer norms on a stream that the caller names, beside another
current one; rows that are no numbers through every activation and kernel."""
import pytest

torch = pytest.importorskip("torch")

import quantized_moe_expert_top_amd as moe  # noqa: E402
from test_int8_ops import ACTS, BF, DEV, F32, gen, make_layer, randn, scales, weights  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [3, 40, 300])
def test_named_stream(T):
    """Inputs are made on the named stream, behind work that holds it up, and read there:
    a call on any other stream would read them before they are written."""
    H, I, E, k = 512, 256, 32, 4
    p = make_layer(T, H, I, E, T)
    w, b = randn(gen(1), (H,), BF), randn(gen(2), (H,), BF)
    e = lambda *s, t=BF: torch.empty(s, dtype=t, device=DEV)  # noqa: E731
    n = moe.layer_w8a8_workspace(T, H, I, E, k)

    def outputs():
        return dict(h=e(T, H), q=e(T, H, t=torch.int8), qs=e(T, t=F32), y=e(T, 2 * I), ids=e(T, k, t=torch.int32),
                    w=e(T, k, t=F32), out=e(T, H), dr=e(T, H), dw=e(H, t=F32), db=e(H, t=F32),
                    ws=e(n, t=torch.uint8), lws=e(moe.linear_w8a8_workspace(T, H), t=torch.uint8),
                    nws=e(moe.layer_norm_backward_workspace(T, H), t=torch.uint8))

    def calls(x, o, stream=None):
        moe.layer_norm(x, w, o["h"], b=b, stream=stream)
        moe.quant_rows(o["h"], o["q"], o["qs"], stream=stream)
        moe.linear_w8a8(o["h"], p["w13"][0], p["s13"][0], o["y"], ws=o["lws"], stream=stream)
        moe.layer_w8a8(p["logits"], o["h"], p["w13"], p["s13"], p["w2"], p["s2"], o["ids"], o["w"], o["out"],
                       o["ws"], stream=stream)
        moe.layer_norm_backward(x, w, o["out"], o["dr"], dw=o["dw"], db=o["db"], ws=o["nws"], stream=stream)

    want, got = outputs(), outputs()
    calls(p["x"], want)
    x = torch.zeros_like(p["x"])
    side, big = torch.cuda.Stream(), torch.randn((4096, 4096), device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(8):
            big = big @ big
            big /= big.norm()
        x.copy_(p["x"])
    calls(x, got, stream=side.cuda_stream)
    side.synchronize()
    for name in ("h", "q", "qs", "y", "ids", "w", "out", "dr", "dw", "db"):
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [3, 16, 40, 300])
def test_rows_that_are_no_numbers(M, act):
    """NaN through every activation and the residual; no bit of another row changes."""
    K, N = 8208 if M == 16 else 528, 48      # 16 rows: the kernel without rings
    g = gen(M)
    x, w, u = randn(g, (M, K), BF), weights(g, (N, K)), scales(g, (N,), K)
    No = N // 2 if act == "swiglu" else N
    r = randn(g, (M, No), F32)
    ws = torch.empty(moe.linear_w8a8_workspace(M, K), dtype=torch.uint8, device=DEV)
    good, y = torch.empty((M, No), device=DEV), torch.empty((M, No), device=DEV)
    moe.linear_w8a8(x, w, u, good, residual=r, act=act, ws=ws)
    x[0, K - 1], x[M - 1, 5] = float("nan"), float("-inf")
    moe.linear_w8a8(x, w, u, y, residual=r, act=act, ws=ws)
    assert torch.isnan(y[0]).all() and torch.isnan(y[M - 1]).all()
    assert torch.equal(y[1:M - 1], good[1:M - 1])
