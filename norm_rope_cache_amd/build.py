"""Build libnrc.so (the HIP library behind include/nrc.h) for gfx950, in-tree.

    python -m norm_rope_cache_amd.build

Every source is compiled ahead of time with hipcc; nothing is JIT-compiled at
run time. Floating-point flags: no contraction (an FMA only where the source
writes one), no fast math, f32 subnormals kept, correctly rounded f32 divide
and sqrt, and no packed-FP32 instructions.
"""

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libnrc.so")
SOURCES = ["api.cpp", "context_norms.hip", "norms_ex.hip", "draft_boundary.hip", "kv_project.hip", "kv_store.hip", "selftest.hip",
           "cache_api.cpp", "rope.hip", "tree_attention.hip", "attention_mass.hip", "kv_evict.hip"]
# the chain's kernels and the entry points that choose among them: what the stored counter measurements were taken of
CHAIN_SOURCES = ["api.cpp", "context_norms.hip", "device_common.h", "draft_boundary.hip", "kernels.h", "kv_project.hip",
                 "kv_store.hip", "norms_ex.hip", "selftest.hip", "status.h"]

ARCH = "gfx950"
COMMON = [
    "-O3",
    "-std=c++17",
    "-fPIC",
    f"--offload-arch={ARCH}",
    "-ffp-contract=off",
    "-fno-fast-math",
    "-fno-gpu-flush-denormals-to-zero",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Xclang",
    "-target-feature",
    "-Xclang",
    "-packed-fp32-ops",
    "-Wall",
]


def hipcc():
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _compile(src):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [hipcc(), *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the packed-fp32 feature and says so; drop that line
    noise = "'-packed-fp32-ops' is not a recognized feature"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def _code_only(text):
    """C/C++ source with comments removed and whitespace runs collapsed
    (string and character literals kept as written)."""
    out, i, n = [], 0, len(text)
    while i < n:
        c = text[i]
        if c in "\"'":
            j = i + 1
            while j < n and text[j] != c:
                j += 2 if text[j] == "\\" else 1
            out.append(text[i:j + 1])
            i = j + 1
        elif text.startswith("//", i):
            j = text.find("\n", i)
            i = n if j < 0 else j
        elif text.startswith("/*", i):
            j = text.find("*/", i + 2)
            i = n if j < 0 else j + 2
        else:
            out.append(c)
            i += 1
    return " ".join("".join(out).split())


def source_hash():
    """Hash of the chain's sources and headers, kernels and entry points, with
    comments and layout removed (identifies what a stored counter measurement
    belongs to; a change to comments or to other operators keeps it)."""
    import hashlib

    h = hashlib.sha256()
    for name in CHAIN_SOURCES:
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            h.update(name.encode() + b"\0" + _code_only(f.read()).encode())
    return h.hexdigest()[:16]


def build():
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build())
