"""Buffers of the W8A8 layer: what each way through it holds, and the whole layer on buffers
whose workspace it makes itself."""
import pytest

torch = pytest.importorskip("torch")

import quantized_moe_expert_top_amd as moe  # noqa: E402

try:
    moe.load()
    BUILT = True
except RuntimeError:
    BUILT = False

pytestmark = pytest.mark.skipif(not BUILT, reason="libmoe.so not built")


def test_separate_calls_hold_no_workspace_of_the_whole_layer():
    b = moe.LayerBuffers.alloc(64, 256, 128, 16, 4, "w8a8", device="cpu")
    assert b.layer_ws.nbytes == 16
    a = moe.LayerBuffers.alloc(2, 256, 128, 16, 4, "w4a16", device="cpu")
    assert a.layer_ws.nbytes >= moe._lib.layer_w4a16_workspace(2, 256, 128, 16, 4) > 16


def test_whole_layer_makes_its_workspace_once(monkeypatch):
    seen = []
    monkeypatch.setattr(moe, "layer_w8a8", lambda *a, **k: seen.append(a[9]))
    b = moe.LayerBuffers.alloc(5, 256, 128, 16, 4, "w8a8", device="cpu")
    x = torch.zeros((5, 256), dtype=torch.int16)
    for _ in range(2):
        moe.moe_layer(b, x, None, (None,) * 4)
    assert seen[0] is seen[1] is b.layer_ws
    assert b.layer_ws.nbytes == moe.layer_w8a8_workspace(5, 256, 128, 16, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0, 2, 40])
def test_first_call_in_a_capture(T):
    """The workspace made inside a captured call serves its replays and eager calls."""
    H, I, E, k = 256, 128, 16, 4
    g = torch.Generator(device="cuda").manual_seed(T)
    i8 = dict(generator=g, device="cuda", dtype=torch.int8)
    w13, w2 = torch.randint(-128, 128, (E, 2 * I, H), **i8), torch.randint(-128, 128, (E, H, I), **i8)
    s13, s2 = torch.rand((E, 2 * I), device="cuda") * 1e-3, torch.rand((E, H), device="cuda") * 1e-3
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    logits = torch.randn((T, E), generator=g, device="cuda")
    want = moe.moe_layer(moe.LayerBuffers.alloc(T, H, I, E, k, "w8a8"), x, logits, (w13, s13, w2, s2)).clone()
    b = moe.LayerBuffers.alloc(T, H, I, E, k, "w8a8")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_layer(b, x, logits, (w13, s13, w2, s2))
    for _ in range(3):
        b.out.fill_(7.0)
        b.offsets.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.out, want) and int(b.offsets[E]) == T * k and int(b.offsets[0]) == 0
        b.out.fill_(7.0)
        moe.moe_layer(b, x, logits, (w13, s13, w2, s2))
        torch.cuda.synchronize()
        assert torch.equal(b.out, want)


@pytest.mark.gpu
def test_first_call_on_a_named_stream():
    """The workspace comes from that stream's memory, not from what the current stream freed
    last and may still be using."""
    T, H, I, E, k = 5, 256, 128, 16, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    i8 = dict(generator=g, device="cuda", dtype=torch.int8)
    weights = (torch.randint(-128, 128, (E, 2 * I, H), **i8), torch.rand((E, 2 * I), device="cuda") * 1e-3,
               torch.randint(-128, 128, (E, H, I), **i8), torch.rand((E, H), device="cuda") * 1e-3)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    logits = torch.randn((T, E), generator=g, device="cuda")
    want = moe.moe_layer(moe.LayerBuffers.alloc(T, H, I, E, k, "w8a8"), x, logits, weights).clone()
    b, side = moe.LayerBuffers.alloc(T, H, I, E, k, "w8a8"), torch.cuda.Stream()
    freed = torch.empty(moe.layer_w8a8_workspace(T, H, I, E, k), dtype=torch.uint8, device="cuda")
    at = freed.data_ptr()
    torch.cuda.synchronize()
    del freed
    out = moe.moe_layer(b, x, logits, weights, stream=side.cuda_stream)
    side.synchronize()
    assert b.layer_ws.data_ptr() != at
    assert torch.equal(out, want)
    b = moe.LayerBuffers.alloc(T, H, I, E, k, "w8a8")
    assert torch.equal(moe.moe_layer(b, x, logits, weights, stream=0), want)   # the default stream by number
