"""Builds the HIP library libsegtopk.so for gfx950 with hipcc (in-tree).

Every HIP source under csrc/ (the host code and one kernel unit per key type) and
csrc_ops/ (the operators around the selection) is compiled to an object in
parallel, then the objects are linked into one shared library.  Objects go to a
build folder beside the sources.  The operators' binding for torch tensors
(csrc_ops/binding.cpp) is host code, built by g++ as the extension module
_binding.so.  The benchmark's stream-read probe (probe/stream_read.hip) is built alongside as
libsegtopk_probe.so; the top-k library does not use it.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
# Apart from the selection's sources, which the benchmark's traffic figures are tied to.
CSRC_OPS = os.path.join(HERE, "csrc_ops")
OBJ_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libsegtopk.so")
PROBE_SRC = os.path.join(HERE, "probe", "stream_read.hip")
PROBE_LIB = os.path.join(HERE, "probe", "libsegtopk_probe.so")
BINDING_SRC = os.path.join(CSRC_OPS, "binding.cpp")
BINDING_LIB = os.path.join(HERE, "_binding.so")
ARCH = os.environ.get("SEGTOPK_OFFLOAD_ARCH", "gfx950")

HIPCC_FLAGS = [
    "-O3", "-std=c++17", "-fPIC",
    f"--offload-arch={ARCH}",
    # Keep the compiler from forming packed-fp32 instructions.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def sources() -> list:
    return [s for folder in (CSRC, CSRC_OPS) for s in sorted(glob.glob(os.path.join(folder, "*.hip")))]


def binding_command(out: str) -> list:
    import torch
    base = os.path.dirname(torch.__file__)
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", "-I", os.path.join(ROOT, "include"),
            "-isystem", os.path.join(base, "include"),
            "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
            "-isystem", "/opt/rocm/include", "-isystem", sysconfig.get_paths()["include"],
            BINDING_SRC, "-o", out, "-L", os.path.join(base, "lib"),
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip"]


def build(verbose: bool = False, jobs: int | None = None) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    os.makedirs(OBJ_DIR, exist_ok=True)
    srcs = sources()
    objs = [os.path.join(OBJ_DIR, os.path.basename(s)[:-4] + ".o") for s in srcs]
    cmds = [[hipcc, *HIPCC_FLAGS, "-c", s, "-o", o] for s, o in zip(srcs, objs)]
    # The benchmark's stream-read probe: a library of its own.
    cmds.append([hipcc, *HIPCC_FLAGS, "-shared", PROBE_SRC, "-o", PROBE_LIB])

    def run(c):
        if verbose:
            print(" ".join(c), flush=True)
        return subprocess.run(c, capture_output=True, text=True)

    def check(r):
        if r.stderr and verbose:
            # hipcc's host pass warns about the device-only feature flag.
            lines = [ln for ln in r.stderr.splitlines() if "packed-fp32-ops" not in ln]
            if lines:
                print("\n".join(lines), flush=True)
        if r.returncode != 0:
            raise subprocess.CalledProcessError(r.returncode, r.args, r.stdout, r.stderr)

    jobs = jobs or min(len(cmds) + 1, max(1, min(16, os.cpu_count() or 1)))
    with ThreadPoolExecutor(jobs) as ex:
        # The C library needs hipcc alone, and is linked whatever comes of the binding.
        binding = ex.submit(lambda: run(binding_command(BINDING_LIB + ".tmp")))
        for r in ex.map(run, cmds):
            check(r)
        tmp = LIB + ".tmp"
        link = [hipcc, "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp]
        if verbose:
            print(" ".join(link), flush=True)
        subprocess.check_call(link)
        os.replace(tmp, LIB)
        check(binding.result())
    os.replace(BINDING_LIB + ".tmp", BINDING_LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
