"""The C library is built by hipcc alone: what keeps the Python binding from being
built (no torch, no g++) does not keep libmoe.so from being linked."""
import os
import stat
import sys

import pytest

from quantized_moe_expert_top_amd import build

# stands for hipcc: writes its output file and the remarks that the build reads
HIPCC = """#!/bin/sh
while [ $# -gt 0 ]; do
  if [ "$1" = "-o" ]; then echo built > "$2"; fi
  shift
done
echo "a.hip:1:1: remark: Function Name: k [-Rpass-analysis=kernel-resource-usage]" >&2
echo "a.hip:1:1: remark:     ScratchSize [bytes/lane]: 0 [-Rpass-analysis=kernel-resource-usage]" >&2
"""


@pytest.fixture
def places(tmp_path, monkeypatch):
    fake = tmp_path / "hipcc"
    fake.write_text(HIPCC)
    fake.chmod(fake.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("HIPCC", str(fake))
    monkeypatch.setattr(build, "OBJDIR", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libmoe.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_block_binding.so"))
    return tmp_path


def test_library_without_torch(places, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)       # its import raises ImportError
    assert build.build(verbose=True) == str(places / "libmoe.so")
    assert os.path.exists(places / "libmoe.so")
    assert not os.path.exists(places / "_block_binding.so")
    assert "torch" in capsys.readouterr().out


def test_library_is_linked_before_a_failing_binding_is_reported(places, monkeypatch):
    monkeypatch.setenv("CXX", "/bin/false")
    with pytest.raises(RuntimeError, match="block_binding"):
        build.build()
    assert os.path.exists(places / "libmoe.so")
