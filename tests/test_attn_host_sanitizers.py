"""The host code of the attention operators under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU): moe_attn.hip is built a second time with
host-only instrumentation (its gfx950 code as usual), linked with the ordinary
object of the rest of the library, and the C-ABI checks of test_attn_abi.py run
against it in a child process that preloads the sanitizer runtime.

The build goes to _build/asan_attn/ and is reused while the sources hash to the
value stamped beside it."""
import hashlib
import os
import subprocess
import sys

import pytest

from test_host_sanitizers import DRIVER, ROOT, _asan_runtime

OUT = os.path.join(ROOT, "_build", "asan_attn")
LIB = os.path.join(OUT, "libmoe_mlp.so")
STAMP = os.path.join(OUT, "sources.sha256")


def _digest():
    csrc, inc = os.path.join(ROOT, "routed_expert_mlp_amd", "csrc"), os.path.join(ROOT, "include")
    h = hashlib.sha256()
    for d in (csrc, inc):
        for f in sorted(os.listdir(d)):
            with open(os.path.join(d, f), "rb") as src:
                h.update(f.encode() + b"\0" + src.read())
    return h.hexdigest()


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]


def _build(hipcc):
    digest = _digest()
    if os.path.exists(LIB) and os.path.exists(STAMP) and open(STAMP).read().strip() == digest:
        return
    from routed_expert_mlp_amd import build as B
    os.makedirs(OUT, exist_ok=True)
    flags = [f for f in B.HIPCC_FLAGS if f not in ("-Wall", "-shared")] + ["-I", os.path.join(ROOT, "include"), "-c"]
    host = ["-O1", "-g", "-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
            "-fno-omit-frame-pointer"]
    attn, rest = os.path.join(OUT, "moe_attn.o"), os.path.join(B.LIB_DIR, "moe_mlp.o")
    _run([hipcc] + flags + [x for f in host for x in ("-Xarch_host", f)] + [B.ATTN_SRC, "-o", attn])
    if not os.path.exists(rest):
        rest = os.path.join(OUT, "moe_mlp.o")
        _run([hipcc] + flags + [B.SRC, "-o", rest])
    link = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-shared-libsan"]
    _run([hipcc, "--offload-arch=gfx950", "-fPIC", "-shared"] + link + [rest, attn, "-o", LIB + ".tmp"])
    os.replace(LIB + ".tmp", LIB)
    with open(STAMP, "w") as f:
        f.write(digest + "\n")


@pytest.mark.slow
def test_attn_abi_checks_under_host_asan_ubsan():
    from routed_expert_mlp_amd import build as B
    try:
        hipcc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    rt = _asan_runtime(hipcc)
    if rt is None:
        pytest.skip("no shared ASan runtime next to hipcc")
    _build(hipcc)
    syms = subprocess.run(["nm", "-D", "--undefined-only", LIB], capture_output=True, text=True).stdout
    assert "__asan_report" in syms and "__ubsan_handle" in syms
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-c", DRIVER, ROOT, LIB, os.path.join(ROOT, "tests", "test_attn_abi.py")],
                       capture_output=True, text=True, env=env, timeout=600)
    out = r.stdout[-3000:] + r.stderr[-3000:]
    assert r.returncode == 0, out
    assert "passed" in r.stdout and "ERROR: AddressSanitizer" not in out and "runtime error" not in out, out
