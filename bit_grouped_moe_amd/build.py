"""Build libgq.so (HIP kernels + C ABI), libgq_probes.so (benchmark
controls) and _calls.so (host code: the binding's short calls) in-tree for
gfx950.

    python -m bit_grouped_moe_amd.build        # or __graft_entry__.build()

Each .hip source is compiled to an object with hipcc, then linked into
``bit_grouped_moe_amd/libgq.so``.  Always rebuilds.
"""

import hashlib
import os
import re
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgq.so")
PROBE_LIB = os.path.join(HERE, "libgq_probes.so")
PROBE_SRC = os.path.join(CSRC, "probes", "probes.hip")
CALLS_LIB = os.path.join(HERE, "_calls.so")
CALLS_SRC = os.path.join(CSRC, "binding", "calls.cpp")
HEADER = os.path.join(os.path.dirname(HERE), "include", "gq.h")
ARCH = "gfx950"

CFLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # no packed-FP32 VALU ops (v_pk_*_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # keep float32 denormals (exact e8m0 scaling of tiny weights)
    "-fno-gpu-flush-denormals-to-zero",
    # kernel arguments preloaded into SGPRs by the dispatcher (up to 16
    # dwords; the code keeps a fallback that loads them itself): saves one
    # dependent load at the start of every kernel, ~0.3 us per decode GEMV
    "-mllvm", "-amdgpu-kernarg-preload-count=16",
    "-Wall", "-Wno-unused-command-line-argument",
]


def _hipcc():
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    raise RuntimeError("hipcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def build(verbose=False, jobs=8):
    os.makedirs(BUILD, exist_ok=True)
    hipcc = _hipcc()
    srcs = sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-4] + ".o")
        cmd = [hipcc, *CFLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        out = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                        if "packed-fp32-ops" not in l)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed for {src}:\n{out}")
        if verbose and out.strip():
            print(out, file=sys.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=jobs) as ex:
        calls = ex.submit(build_calls)
        objs = list(ex.map(compile_one, srcs))
    link(hipcc, objs, LIB)
    link(hipcc, [compile_one(PROBE_SRC)], PROBE_LIB)
    try:
        calls.result()
    except (ImportError, OSError, RuntimeError) as e:
        # every call works without them, through Python code; an earlier
        # build's module may not fit this library
        print(f"short calls not built, the Python code makes every call: {e}", file=sys.stderr)
        if os.path.exists(CALLS_LIB):
            os.remove(CALLS_LIB)
    return LIB


def header_id():
    """What include/gq.h declares, without its comments and spacing, as a
    short text: the short calls hold it and are used with that header only."""
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return hashlib.sha256(" ".join(text.split()).encode()).hexdigest()[:16]


def build_calls():
    """The binding's short calls, against the installed torch (host code)."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    tmp = CALLS_LIB + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D__HIP_PLATFORM_AMD__", f'-DGQ_TORCH_VERSION="{torch.__version__}"',
           f'-DGQ_HEADER_ID="{header_id()}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"),
           "-isystem", sysconfig.get_paths()["include"], CALLS_SRC, "-o", tmp,
           "-L" + os.path.join(root, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {CALLS_SRC}:\n{r.stdout}{r.stderr}")
    os.replace(tmp, CALLS_LIB)


def link(hipcc, objs, lib):
    tmp = lib + ".tmp"
    cmd = [hipcc, "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, lib)


if __name__ == "__main__":
    print(build(verbose=True))
