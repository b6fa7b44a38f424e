"""The compiled pipelines of the block products (CPU: hipcc cross-compiles).

The tile kernels count their loads to LDS by hand: between the first and the last
MFMA of a kernel the only waits on vector memory may be the hand-written ones. The
compiler adds one before an LDS read whenever it cannot tell that the read does
not need the loads in flight, and each such wait empties the pipeline (8192 x
4096 x 7168: 464 us with them, 376 without)."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def assembly(source):
    from quantized_moe_expert_top_amd import build
    try:
        hipcc = build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    r = subprocess.run([hipcc, *build.FLAGS, "--cuda-device-only", "-S",
                        os.path.join(build.CSRC, source), "-o", "-"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


def stray_waits(text, kernel):
    """{symbol: waits on vector memory between its MFMAs that no asm block wrote}"""
    found = {}
    for m in re.finditer(r"^(_Z\w*%s\w*):\s*;? ?@?.*?^\s*s_endpgm" % kernel, text, re.S | re.M):
        lines = m.group(0).splitlines()
        mfma = [i for i, ln in enumerate(lines) if "v_mfma_" in ln]
        assert mfma, m.group(1)
        bad, by_hand = [], False
        for ln in lines[mfma[0]:mfma[-1]]:
            if "ASMSTART" in ln:
                by_hand = True
            elif "ASMEND" in ln:
                by_hand = False
            elif "vmcnt" in ln and not by_hand:
                bad.append(ln.strip())
        found[m.group(1)] = bad
    return found


@pytest.mark.parametrize("source,kernels", [("mm_nt.hip", 12), ("mm_nn.hip", 12)])
def test_no_waits_but_the_counted_ones(source, kernels):
    found = stray_waits(assembly(source), "mm_kernel")
    assert len(found) == kernels, sorted(found)
    assert not any(found.values()), {k: v for k, v in found.items() if v}


def test_stray_wait_is_seen():
    text = ("_Z9mm_kernelv:\n v_mfma_f32 a\n ;;#ASMSTART\n s_waitcnt vmcnt(4)\n ;;#ASMEND\n"
            "{} ds_read_b128 b\n v_mfma_f32 c\n s_waitcnt vmcnt(0)\n s_endpgm\n")
    assert stray_waits(text.format(""), "mm_kernel") == {"_Z9mm_kernelv": []}
    assert stray_waits(text.format(" s_waitcnt vmcnt(0)\n"), "mm_kernel") == {
        "_Z9mm_kernelv": ["s_waitcnt vmcnt(0)"]}
