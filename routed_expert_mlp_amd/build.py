"""Build the HIP library in-tree: routed_expert_mlp_amd/lib/libmoe_mlp.so (gfx950).

    python -m routed_expert_mlp_amd.build
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "moe_mlp.hip")
ATTN_SRC = os.path.join(HERE, "csrc", "moe_attn.hip")
LIB_DIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIB_DIR, "libmoe_mlp.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # keep packed fp32 vector instructions out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def hipcc():
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    raise RuntimeError("hipcc not found")


def build(verbose=False):
    """Compile both sources side by side and link them into LIB; no object stays behind, of which one could be
    linked into something else after its sources have changed."""
    os.makedirs(LIB_DIR, exist_ok=True)
    objs = [os.path.join(LIB_DIR, os.path.basename(src)[:-4] + ".o") for src in (SRC, ATTN_SRC)]
    try:
        return _build([hipcc()] + HIPCC_FLAGS, objs, verbose)
    finally:
        for obj in objs:
            if os.path.exists(obj):
                os.remove(obj)


def _build(base, objs, verbose):
    jobs = []
    for src, obj in zip((SRC, ATTN_SRC), objs):
        cmd = [f for f in base if f != "-shared"] + ["-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        jobs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    tmp = LIB + ".tmp"
    outputs = [job.communicate()[0] for job in jobs]
    for job, output in zip(jobs, outputs):
        _check(output, job.returncode, verbose)
    cmd = [base[0], "--offload-arch=gfx950", "-fPIC", "-shared"] + objs + ["-o", tmp]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    _check(r.stdout, r.returncode, verbose)
    os.replace(tmp, LIB)
    return LIB


def _check(output, status, verbose):
    err = "\n".join(l for l in output.splitlines() if "packed-fp32-ops" not in l)
    if status != 0:
        raise RuntimeError(f"hipcc failed ({status}):\n{err}")
    if err.strip() and verbose:
        print(err, file=sys.stderr)


if __name__ == "__main__":
    print(build(verbose=True))
