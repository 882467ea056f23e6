"""Where the library's build keeps its objects while it runs: not where other builds look for them."""
import os
import stat

from routed_expert_mlp_amd import build as B

COMPILER = """#!/bin/sh
for last; do :; done
ls "%s" >> "%s"
echo built > "$last"
"""


def test_no_object_stands_beside_the_library_while_it_is_built(tmp_path, monkeypatch):
    """A build that is killed has no chance to remove its objects: there are none, then, whose sources may have changed
    by the time that another build links them."""
    hipcc, lib, seen = tmp_path / "hipcc", tmp_path / "lib", tmp_path / "seen"
    hipcc.write_text(COMPILER % (lib, seen))
    hipcc.chmod(hipcc.stat().st_mode | stat.S_IXUSR)
    lib.mkdir()
    (lib / "moe_mlp.o").write_text("of another day")
    monkeypatch.setattr(B, "hipcc", lambda: str(hipcc))
    monkeypatch.setattr(B, "LIB_DIR", str(lib))
    monkeypatch.setattr(B, "LIB", str(lib / "libmoe_mlp.so"))
    B.build()
    assert os.path.exists(lib / "libmoe_mlp.so")
    assert not [f for f in seen.read_text().split() if f.endswith(".o")]
