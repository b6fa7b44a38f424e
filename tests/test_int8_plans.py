"""Every kernel that int8 products and the W8A8 layer are dispatched to, named by the
dispatch itself: products with every activation, type and operand of their epilogue, on
codes and on values; the layer on every way, depth of rings and tile."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import quantized_moe_expert_top_amd as moe  # noqa: E402
from test_int8_ops import ACTS, BF, F32, HF, check_layer, gen, make_layer, randn, run_linear  # noqa: E402

try:
    moe.load()
    BUILT = True
except RuntimeError:
    BUILT = False

pytestmark = pytest.mark.skipif(not BUILT, reason="libmoe.so not built")

# (rows, K, N): the kernel, whatever the activation, the depth of its rings, and where the
# codes of values are made. Rows, columns and contraction that tiles and stages do not
# divide.
LINEAR = {(5, 1040, 304): ("rings", 8, "in the launch"), (13, 4112, 304): ("rings", 4, "before it"),
          (16, 8208, 304): ("rows by 16", 0, "before it"), (2, 64, 32784): ("rows by 16", 0, "before it"),
          (61, 2064, 1040): ("rows by 32", 0, "before it"), (301, 1040, 1040): ("64x64", 0, "before it"),
          (8691, 1456, 80): ("64x128", 0, "before it"), (4093, 1040, 1552): ("128x128", 0, "before it"),
          (1219, 10256, 1744): ("128x128 deep", 0, "before it"),
          (9000, 1040, 1552): ("128x256", 0, "before it"), (4171, 2352, 2192): ("256x256", 0, "before it"),
          # where two tiles of 32 rows would take a second round
          (33, 7168, 4112): ("64x64", 0, "before it")}


@pytest.mark.parametrize("M,K,N", LINEAR)
def test_linear_plans(M, K, N):
    kernel, depth, made = LINEAR[M, K, N]
    for act in ACTS:
        assert moe.linear_w8a8_plan(M, K, N, act) == dict(kernel=kernel, depth=depth, codes=made), act
        assert moe.linear_w8a8_plan(M, K, N, act, codes=True) == dict(kernel=kernel, depth=depth, codes=None)


def test_every_kernel_of_products_is_here():
    assert {k for k, _, _ in LINEAR.values()} == {*moe._block._TILES, "rings"}
    assert {d for k, d, _ in LINEAR.values() if k == "rings"} == {8, 4}


def test_linear_plan_refusals():
    lib, s = moe._block._load(), moe._block.MoeW8Shape(4, 64, 32, 3, 0, 0)
    plan = (ctypes.c_int32 * 3)()
    assert lib.moe_linear_w8a8_plan(None, plan) == 1 and lib.moe_linear_w8a8_plan(ctypes.byref(s), None) == 1
    for bad in ((-1, 64, 32), (4, 72, 32), (4, 64, 20)):
        with pytest.raises(moe.MoeError):
            moe.linear_w8a8_plan(*bad)
    assert moe.linear_w8a8_plan(0, 64, 32)["kernel"]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", LINEAR)
@pytest.mark.parametrize("act", ACTS)
def test_linear(M, K, N, act):
    """Given codes, the residual added in place; values, with a bias, to another type."""
    n = ACTS.index(act) + M % 3
    run_linear(M, K, N, act, BF, (F32, HF, BF)[n % 3], n % 2 == 0, True, True, M, in_place=True)
    run_linear(M, K, N, act, (HF, BF)[n % 2], (HF, BF, F32)[n % 3], True, n % 2 == 0, False, M + 1)


HERE, AHEAD = "in the launch", "before it"
# (T, H, I, E, k): the way, then for gate/up and for down the depth of the rings or the
# tiles, and where the codes are made
LAYER = {(2, 528, 272, 24, 6): ("rings", (8, HERE), (8, HERE)),
         (2, 272, 144, 200, 4): ("rings", (8, HERE), (8, HERE)),    # routers of 256 and of
         (3, 272, 144, 1000, 4): ("rings", (8, HERE), (8, HERE)),   # 1024 experts
         (9, 272, 80, 24, 3): ("rings", (8, AHEAD), (8, HERE)),
         (12, 272, 144, 1000, 4): ("rings", (8, AHEAD), (8, HERE)),
         (4, 272, 1200, 12, 4): ("rings", (8, HERE), (8, AHEAD)),
         (16, 2048, 128, 32, 8): ("rings", (4, AHEAD), (4, HERE)),
         (16, 528, 96, 18, 11): ("rings", (8, AHEAD), (4, AHEAD)),
         (13, 7168, 128, 16, 2): ("rings", (2, AHEAD), (8, HERE)),
         (16, 7168, 32, 32, 32): ("rings", (2, AHEAD), (2, HERE)),
         (13, 272, 224, 43, 28): ("rings", (8, AHEAD), (2, AHEAD)),
         (18, 272, 144, 24, 4): ("rings by 16 rows", (4, AHEAD), (4, AHEAD)),
         (18, 144, 80, 1, 1): ("tiles", ("rows by 16", AHEAD), ("rows by 16", AHEAD)),
         (20, 144, 80, 132, 28): ("tiles", ("64x64", AHEAD), ("64x64", AHEAD)),
         (67, 144, 48, 267, 9): ("tiles", ("64x128", AHEAD), ("64x64", AHEAD)),
         (174, 80, 48, 350, 3): ("tiles", ("64x128", AHEAD), ("64x128", AHEAD)),
         (300, 272, 144, 3, 2): ("tiles of the grouped FFN", (None, AHEAD), (None, AHEAD))}


@pytest.mark.parametrize("shape", LAYER)
def test_layer_plans(shape):
    way, up, down = LAYER[shape]
    assert moe.layer_w8a8_plan(*shape) == dict(way=way, gate_up=up, down=down)


def test_every_kernel_of_the_layer_is_here():
    """All that a sweep of the dispatch finds."""
    have = {(w, i, h) for w, *halves in LAYER.values() for i, h in enumerate(halves)}
    for T in (1, 2, 3, 5, 8, 9, 13, 16, 17, 40, 64, 200, 500, 2000):
        for H in (16, 272, 2048, 5600, 7168, 16384):
            for I in (16, 96, 272, 768, 1200, 2048, 16384):
                for E, k in ((1, 1), (3, 2), (16, 4), (64, 32), (128, 8), (1024, 9)):
                    if T * k * max(H, I) >= 2 ** 31 or 2 * H * I >= 2 ** 31:
                        continue
                    p = moe.layer_w8a8_plan(T, H, I, E, k)
                    assert (p["way"], 0, p["gate_up"]) in have and (p["way"], 1, p["down"]) in have, (
                        T, H, I, E, k, p)


def test_layer_plan_refusals():
    lib, s = moe._block._load(), moe._lib.MoeShape(4, 64, 32, 8, 2)
    plan = (ctypes.c_int32 * 5)()
    assert lib.moe_layer_w8a8_plan(None, plan) == 1 and lib.moe_layer_w8a8_plan(ctypes.byref(s), None) == 1
    for bad in ((-1, 64, 32, 8, 2), (4, 72, 32, 8, 2), (4, 64, 32, 8, 9)):
        with pytest.raises(moe.MoeError):
            moe.layer_w8a8_plan(*bad)
    assert moe.layer_w8a8_plan(0, 64, 32, 8, 2)["way"]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", LAYER)
@pytest.mark.parametrize("x_t,out", [(BF, F32), (HF, HF), (HF, BF)])
def test_layer(shape, x_t, out):
    T, H, I, E, k = shape
    p = make_layer(T, H, I, E, T * 5 + H + k, x_t)
    check_layer(p, k, out)
    check_layer(p, k, out, residual=randn(gen(3), (T, H), out), in_place=True)
