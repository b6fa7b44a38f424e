"""The compiled pipelines of all tile kernels of the block products, read to each
kernel's end (CPU: hipcc cross-compiles).

Loads to LDS are waited for by count, by hand. Inside a loop of stages (an innermost
loop that multiplies) no other wait on vector memory may stand: the compiler's own
would be for every load in flight, and empty the pipeline."""
import re

import pytest

from test_block_build import assembly


def functions(text, kernel):
    """{symbol: its lines, to the function's end}"""
    return {m.group(1): m.group(0).splitlines()
            for m in re.finditer(r"^(_Z\w*%s\w*):.*?^\.Lfunc_end\d+:" % kernel, text, re.S | re.M)}


def stage_loops(lines):
    """[first, last] lines of the innermost loops that hold an MFMA: from a label to
    the last branch back to it."""
    label = {m.group(1): i for i, ln in enumerate(lines) if (m := re.match(r"^(\.LBB\w+):", ln))}
    loops = {}
    for i, ln in enumerate(lines):
        m = re.match(r"^\s+s_c?branch\w*\s+(\.LBB\w+)", ln)
        if m and label.get(m.group(1), i) < i:
            loops[label[m.group(1)]] = i
    loops = [(a, b) for a, b in loops.items() if any("v_mfma_" in ln for ln in lines[a:b])]
    return [(a, b) for a, b in loops
            if not any((c, d) != (a, b) and a <= c and d <= b for c, d in loops)]


def waits(lines):
    """(hand-written, other) waits on vector memory"""
    hand, other, by_hand = [], [], False
    for ln in lines:
        if "ASMSTART" in ln:
            by_hand = True
        elif "ASMEND" in ln:
            by_hand = False
        elif "vmcnt" in ln:
            (hand if by_hand else other).append(ln.strip())
    return hand, other


# Two loops of stages in each kernel, with a stage to request and the last ones
# without; twice that where a kernel holds both products.
@pytest.mark.parametrize("source,kernel,count", [
    ("mm_nt.hip", "mm_kernel", 12), ("mm_nn.hip", "mm_kernel", 12), ("mm_tn.hip", "mm_kernel", 8),
    ("mm_pair.hip", "mm_pair_kernel", 4)])
def test_stage_loops_wait_by_count_only(source, kernel, count):
    found = functions(assembly(source), kernel)
    assert len(found) == count, sorted(found)
    for name, lines in found.items():
        loops = stage_loops(lines)
        assert len(loops) >= (4 if kernel == "mm_pair_kernel" else 2), (name, loops)
        for a, b in loops:
            hand, other = waits(lines[a:b])
            assert hand and not other, (name, a, b, hand, other)


def test_a_planted_wait_is_seen():
    text = ("_Z9mm_kernelv:\n s_waitcnt vmcnt(0)\n s_endpgm\n.LBB0_1:\n v_mfma_f32 a\n"
            " ;;#ASMSTART\n s_waitcnt vmcnt(4)\n ;;#ASMEND\n{} s_cbranch_scc1 .LBB0_1\n"
            " s_waitcnt vmcnt(0)\n s_branch .LBB0_0\n s_endpgm\n.Lfunc_end0:\n")
    for planted in ("", " s_waitcnt vmcnt(0)\n"):
        lines = functions(text.format(planted), "mm_kernel")["_Z9mm_kernelv"]
        loops = stage_loops(lines)
        assert len(loops) == 1
        hand, other = waits(lines[slice(*loops[0])])
        assert hand == ["s_waitcnt vmcnt(4)"]
        assert other == ([planted.strip()] if planted else [])
