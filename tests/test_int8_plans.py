"""Every kernel that int8 products are dispatched to, named by the dispatch itself, with
every activation, type and operand of its epilogue, on codes and on values."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import quantized_moe_expert_top_amd as moe  # noqa: E402
from test_int8_ops import ACTS, BF, F32, HF, run_linear  # noqa: E402

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
