"""The compiled pipelines of the int8 kernels (CPU: hipcc cross-compiles). Loads to LDS are
waited for by count, by hand: a loop that multiplies holds no other wait on vector memory,
which would be for every load in flight. The kernel whose rows come to registers leaves
the counting to the compiler; there no wait of the loop is for all loads."""
import re

import pytest

from test_block_build import assembly
from test_block_waits import functions, stage_loops, waits


# how many kernels, and how many such loops each has
@pytest.mark.parametrize("source,kernel,count,loops", [
    ("mm_i8.hip", "mm_kernel", 12, 2), ("mm_i8.hip", "linear_few_kernel", 18, 1),
    ("layer_w8a8.hip", "layer_few_kernel", 39, 1), ("layer_w8a8.hip", "layer_rows_kernel", 2, 1)])
def test_loops_of_products_wait_by_count_only(source, kernel, count, loops):
    found = functions(assembly(source), kernel)
    assert len(found) == count, sorted(found)
    for name, lines in found.items():
        at = stage_loops(lines)
        assert len(at) == loops, (name, at)
        for a, b in at:
            hand, other = waits(lines[a:b])
            assert hand and not other, (name, a, b, hand, other)


def test_rows_in_registers_never_wait_for_all_loads():
    found = functions(assembly("mm_i8.hip"), "mm_few_kernel")
    assert len(found) == 4, sorted(found)
    for name, lines in found.items():
        at = stage_loops(lines)
        assert at, name
        for a, b in at:
            hand, other = waits(lines[a:b])
            assert other and not hand, (name, hand)
            assert all(int(re.search(r"vmcnt\((\d+)\)", w).group(1)) >= 4 for w in other), (name, other)
