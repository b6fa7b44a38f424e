"""Results of MFMAs that inline assembly reads (CPU: hipcc cross-compiles). The compiler
keeps an MFMA's result from being read too early only by instructions that it knows: an asm
block that reads one has to be behind wait states of its own."""
import re

import pytest

from test_block_build import assembly
from test_block_waits import functions

# passes + 3, one more from 4 passes on: 16 passes (32x32 results) need 20
WAIT_STATES = 20
PASSES = {"v_mfma_i32_16x16x64_i8": 4, "v_mfma_f32_16x16x32_bf16": 4, "v_mfma_f32_16x16x32_f16": 4}


def registers(text):
    """VGPRs named in an operand list"""
    out = set()
    for a, b, c in re.findall(r"\bv(?:\[(\d+):(\d+)\]|(\d+))", text):
        out |= set(range(int(a), int(b) + 1)) if a else {int(c)}
    return out


def early_reads(lines):
    """asm instructions that read an MFMA's result before its wait states have passed, in
    the order of the text (a branch only leaves more of them out)"""
    bad, by_hand = [], False
    pending = {}   # register -> wait states left
    for ln in lines:
        if "ASMSTART" in ln:
            by_hand = True
            continue
        if "ASMEND" in ln:
            by_hand = False
            continue
        m = re.match(r"^\s+([a-z]\w+)\s*(.*?)(?:;.*)?$", ln)
        if not m:
            continue
        op, args = m.groups()
        if by_hand and registers(args) & set(pending):
            bad.append(ln.strip())
        states = int(args) + 1 if op == "s_nop" else 1
        pending = {r: n - states for r, n in pending.items() if n > states}
        if op.startswith("v_mfma_"):
            dst = registers(args.split(",")[0])
            need = PASSES[op] + 4 if op in PASSES else WAIT_STATES
            pending.update({r: need for r in dst})
        elif op.startswith("v_") and args:
            for r in registers(args.split(",")[0]):
                pending.pop(r, None)
    return bad


@pytest.mark.parametrize("source", ["mm_i8.hip", "layer_w8a8.hip"])
def test_asm_reads_settled_results(source):
    found = functions(assembly(source), "kernel")
    assert found
    bad = {name: early_reads(lines) for name, lines in found.items()}
    assert not any(bad.values()), {k: v for k, v in bad.items() if v}


@pytest.mark.parametrize("between,seen", [("", True), (" s_nop 6\n", True), (" s_nop 7\n", False),
                                          (" s_nop 3\n s_nop 3\n", False), (" v_mov_b32_e32 v2, 0\n", False)])
def test_a_planted_early_read_is_seen(between, seen):
    text = (" v_mfma_i32_16x16x64_i8 v[2:5], v[6:9], v[14:17], v[2:5]\n" + between +
            " ;;#ASMSTART\n ds_add_u32 v6, v2\n ;;#ASMEND\n")
    assert bool(early_reads(text.splitlines())) == seen
