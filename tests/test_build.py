"""The library's build without a compiler: what it leaves behind."""
import os
import stat

import pytest

from routed_expert_mlp_amd import build as B

COMPILER = """#!/bin/sh
for last; do :; done
echo built > "$last"
case "$*" in *-shared*) exit %d;; esac
"""


@pytest.mark.parametrize("status", [0, 1])
def test_build_leaves_no_objects(tmp_path, monkeypatch, status):
    """Not of this build, whether it links or not, and not of one before: other builds would link them whatever
    sources they are of."""
    hipcc, lib = tmp_path / "hipcc", tmp_path / "lib"
    hipcc.write_text(COMPILER % status)
    hipcc.chmod(hipcc.stat().st_mode | stat.S_IXUSR)
    lib.mkdir()
    (lib / "moe_mlp.o").write_text("of another day")
    monkeypatch.setattr(B, "hipcc", lambda: str(hipcc))
    monkeypatch.setattr(B, "LIB_DIR", str(lib))
    monkeypatch.setattr(B, "LIB", str(lib / "libmoe_mlp.so"))
    if status:
        with pytest.raises(RuntimeError):
            B.build()
    else:
        assert B.build() == str(lib / "libmoe_mlp.so")
        assert os.path.exists(lib / "libmoe_mlp.so")
    assert not [f for f in os.listdir(lib) if f.endswith(".o")]
